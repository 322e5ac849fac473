"""Host side of the evicting cache's calls and of the weight sums (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from tile_routed_mixed_causal_b200 import _lib as L
from tile_routed_mixed_causal_b200 import api
from tile_routed_mixed_causal_b200 import build as tra_build


def test_shape_brings_its_status_word(monkeypatch):
    """The word is there from the start: no call creates it, on whatever stream or in whatever capture
    it runs."""
    s = L.Shape([0, 130, 194], 8, 2, 128, device="cpu")
    for name in ("zeros", "empty", "full", "tensor"):
        monkeypatch.setattr(torch, name, lambda *a, **k: (_ for _ in ()).throw(AssertionError("made late")))
    word = s.status
    assert word.dtype is torch.int32 and word.shape == (1,) and int(word) == 0
    assert s.status.data_ptr() == word.data_ptr()
    assert s.cu_dev.tolist() == [0, 130, 194] and s.cu_dev.is_contiguous()
    assert np.array_equal(s.cu_host, [0, 130, 194])
    assert L.Shape([0, 64], 8, 2, 128, device=None).status is None


def _stub(**kw):
    f = dict(B=2, Hq=8, Hkv=2, d=128, cap=6, n_pool=24)
    f |= {n: 1 << 20 for n in L.PagedCache.NAMES}
    return L._PagedCache(**(f | kw))


@pytest.mark.parametrize("kw", [dict(least=-1), dict(recent=-1), dict(keep=0), dict(keep=7)])
def test_evict_from_refusals(kw):
    tra_build.build()
    a = dict(keep=2, least=100, recent=0) | kw
    assert L.load().paged_cache_evict_from(ctypes.byref(_stub()), a["keep"], a["least"], a["recent"], None, None, None, None,
                                           1 << 20, 1 << 40, 1 << 20, None) == 1


class _Calls:
    """Stands in for the library's calls of a plan: notes which rows each eviction cuts."""

    def __init__(self, monkeypatch):
        self.evicted = []
        monkeypatch.setattr(L, "paged_attention_decode", lambda *a, **k: None)
        monkeypatch.setattr(L, "paged_cache_evict", lambda c, **k: self.evicted.append(k["least"]))


def _plan(**kw):
    tra_build.build()
    return api.EvictingDecodePlan(L.Shape([0, 200, 300, 400], 4, 2, 64, device=None), 2, 4, device="cpu", **kw)


def test_plan_cuts_rows_of_their_own(monkeypatch):
    calls, plan = _Calls(monkeypatch), _plan(per_row=True)
    plan.rows = [[4, 62], [3, 63], [4, 63]]
    plan.step(None, None, None, None)
    assert calls.evicted == [4 * 64 + 63]
    assert plan.rows == [[4, 63], [4, 0], [3, 0]]       # only the last had no room
    plan.step(None, None, None, None)
    assert len(calls.evicted) == 2 and plan.rows == [[3, 0], [4, 1], [3, 1]]


def test_plan_cuts_all_rows_together(monkeypatch):
    calls, plan = _Calls(monkeypatch), _plan()
    plan.rows = [[4, 62], [3, 63], [4, 63]]
    plan.step(None, None, None, None)
    assert calls.evicted == [0]
    assert plan.rows == [[2, 63], [3, 0], [3, 0]]


@pytest.mark.parametrize("per_row", [False, True])
def test_plan_without_a_retired_row(monkeypatch, per_row):
    """A row that is done causes no cut of the others, and is not counted on."""
    calls, plan = _Calls(monkeypatch), _plan(per_row=per_row)
    plan.rows = [[4, 63], [3, 0], [3, 63]]
    plan.cache["state"][:, 0] = 4
    plan.retire(0)
    for _ in range(3):
        plan.step(None, None, None, None)
    assert calls.evicted == [] and plan.rows == [[-1, 63], [3, 3], [4, 2]]
    assert plan.cache["state"][:, 0].tolist() == [-1, 4, 4]


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 2, -2 ** 31 - 1, 10 ** 12])
def test_numbers_past_32_bits(monkeypatch, big):
    """They are refused, not cut off: 2^32 recent tokens are not none."""
    tra_build.build()
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    f32, shape = torch.float32, L.Shape([0, 128], 4, 2, 64, device="cpu")
    cache = L.PagedCache(1, 4, 2, 64, 3, device="cpu")
    monkeypatch.setattr(L, "_launch_device", lambda t: -1)      # as if the tensors were on a GPU
    monkeypatch.setattr(L, "_on", lambda shape, index: None)
    monkeypatch.setattr(L, "_stream", lambda s: None)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(L, "load", lambda: Lib())
    k = z(128, 2, 64)
    with pytest.raises(L.TraError, match="32 bits"):
        L.attention_weight_sums(shape, z(128, 4, 64), k, z(128, 2, t=f32), z(4, 128, t=f32), n_queries=big, softmax_scale=0.1)
    for kw in (dict(keep=big), dict(keep=2, recent=big)):
        with pytest.raises(L.TraError, match="32 bits"):
            L.paged_cache_fill(cache, shape, k, k, **kw)
        with pytest.raises(L.TraError, match="32 bits"):
            L.paged_cache_evict(cache, **kw)
    with pytest.raises(L.TraError, match="32 bits"):
        L.paged_cache_evict(cache, keep=2, least=big)
