"""The evicting cache's calls as a program makes them: on streams of its own, captured, beside other
calls, and with states and pages that are not in order."""
import math

import numpy as np
import pytest
import torch

import tile_routed_mixed_causal_b200 as tra
from tile_routed_mixed_causal_b200 import api

from test_gpu_evicting import DEV, TILE, Mirror, _cu, _filled, _normal, _rng

pytestmark = pytest.mark.gpu


# ================================================================ streams
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_prompt_importance_on_a_stream(handle):
    """The call's own tensors belong to the stream it is given: what the current stream allocates and
    writes right after the call, while that stream has not begun, is not theirs."""
    hq, hkv, d, lens = 8, 2, 128, [700, 130]
    gen, cu = _rng(21), _cu(lens)
    q, k = _normal(gen, cu[-1], hq, d), _normal(gen, cu[-1], hkv, d)
    shape, s = tra.Shape(cu, hq, hkv, d), torch.cuda.Stream()
    want = api.prompt_importance(shape, q, k, n_queries=0)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = api.prompt_importance(shape, q, k, n_queries=0, stream=s.cuda_stream if handle else s)
        other = [torch.full(x, 5.0, device=DEV) for x in ((hq, cu[-1]), (cu[-1], hkv)) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(bool((x == 5.0).all()) for x in other)
        del got, other


def test_plan_on_a_stream():
    """A plan used on a stream of its own from its first call on, its weights dropped at once."""
    hq, hkv, d, lens = 8, 2, 128, [500, 200, 64]
    gen, cu = _rng(23), _cu(lens)
    q, k, v = (_normal(gen, cu[-1], h, d) for h in (hq, hkv, hkv))
    steps = [tuple(_normal(gen, 3, h, d) for h in (hq, hkv, hkv)) for _ in range(3)]
    shape, s = tra.Shape(cu, hq, hkv, d), torch.cuda.Stream()
    torch.cuda.synchronize()
    plans, outs = [], []
    for stream in (None, s):
        if stream is not None:
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)
        plan = api.EvictingDecodePlan(shape, keep=3, limit=5, recent=70)
        plan.prefill(q, k, v, stream=stream)
        other = [torch.full(x, 5.0, device=DEV) for x in ((hq, cu[-1]), (cu[-1], hkv)) for _ in range(4)]
        outs.append([])
        for x in steps:
            outs[-1].append(torch.empty(3, hq, d, dtype=torch.bfloat16, device=DEV))
            plan.step(*x, outs[-1][-1], stream=stream)
        torch.cuda.synchronize()
        assert all(bool((x == 5.0).all()) for x in other)
        plans.append(plan)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for n in plans[0].cache.NAMES:
        assert torch.equal(plans[0].cache[n], plans[1].cache[n]), n
    assert int(plans[1].status) == 0


# ================================================================ the status word of a shape
def test_first_call_in_a_capture():
    """The first call on a shape is a captured one: a replay adds to the shape's status word and clears
    nothing that an earlier call has left there."""
    hq, hkv, d, n = 4, 2, 64, 200
    gen = _rng(31)
    q, k = _normal(gen, n, hq, d), _normal(gen, n, hkv, d)
    w, lse = torch.zeros(n, hkv, device=DEV), torch.zeros(hq, n, device=DEV)
    tra.attention_weight_sums(tra.Shape([0, n], hq, hkv, d), q, k, w, lse, softmax_scale=0.125)     # loads the kernels
    want = w.clone()
    shape = tra.Shape([0, n], hq, hkv, d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=0.125)
    shape.status.fill_(tra.DEV_TIMEOUT)
    w.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert int(shape.status) == tra.DEV_TIMEOUT and torch.equal(w, want)


# ================================================================ page numbers out of range
def _copy(cache):
    return {n: x.clone() for n, x in cache.t.items()}


def _same_row(cache, before, b, names, upto=None):
    for n in names:
        x, y = cache[n][b], before[n][b]
        if upto is not None and n in ("weight", "pos"):
            x, y = x[:, :upto], y[:, :upto]
        assert torch.equal(x, y), n


def _same_pages(cache, before, numbers):
    at = torch.tensor([i for i in numbers if 0 <= i < cache.n_pool], dtype=torch.long, device=DEV)
    for n in ("k8", "v8", "sk", "sv"):
        assert torch.equal(cache[n][at], before[n][at]), n


def _spare(before):
    """A page of the pool that no row has."""
    return min(set(range(before["sk"].shape[0])) - set(before["table"].flatten().tolist()))


OTHERS = ("table", "state", "weight", "pos", "k_tail", "v_tail")


@pytest.mark.parametrize("bad", [-1, 1 << 20, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("entry", [0, 1])
def test_fill_leaves_a_row_with_a_bad_page(bad, entry):
    """One entry of one head: the whole row stays, pages and all; the other row is filled."""
    cache, _ = _filled([(2, 63), (2, 7)], 4, 2, 64, 4, seed=1)
    cache["table"][0, 1, entry] = bad
    gen, cu = _rng(1), [0, 150, 300]
    k, v, w = _normal(gen, 300, 2, 64), _normal(gen, 300, 2, 64), torch.rand(300, 2, generator=gen, device=DEV)
    before, ref = _copy(cache), Mirror(cache)
    ref.t["table"][0, 1, entry] = _spare(before)    # (what the mirror makes of row 0 is not looked at)
    ref.fill(cu, k, v, w, 2, 10)
    tra.paged_cache_fill(cache, tra.Shape(cu, 4, 2, 64), k, v, keep=2, recent=10, weights=w)
    assert int(cache.status) == tra.DEV_BAD_CACHE
    _same_row(cache, before, 0, OTHERS)
    rest = sorted(set(range(cache.n_pool)) - set(cache["table"][1, :, :2].flatten().tolist()))
    _same_pages(cache, before, rest)
    for n in OTHERS:
        assert np.array_equal(cache[n][1].float().cpu().numpy(), ref.t[n][1].astype(np.float32)), n
    at = cache["table"][1, :, :2].flatten().tolist()
    for n in ("k8", "v8", "sk", "sv"):
        assert np.array_equal(cache[n].cpu().numpy()[at], ref.t[n][at]), n


def test_fill_does_not_look_past_its_pages():
    """A number behind the last page that a fill writes is not its business."""
    cache, _ = _filled([(2, 63)], 4, 2, 64, 4, seed=1)
    cache["table"][0, 1, 2:] = -7
    gen = _rng(1)
    k, v = _normal(gen, 150, 2, 64), _normal(gen, 150, 2, 64)
    ref = Mirror(cache)
    tra.paged_cache_fill(cache, tra.Shape([0, 150], 4, 2, 64), k, v, keep=4)
    ref.fill([0, 150], k, v, None, 4, 0)
    assert int(cache.status) == 0
    ref.same()


@pytest.mark.parametrize("recent", [0, 10 ** 6])
@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
@pytest.mark.parametrize("entry,bad", [(0, -1), (2, 1 << 20), (3, 2 ** 31 - 1), (4, -2 ** 31)])
def test_evict_leaves_a_row_with_a_bad_page(entry, bad, apart, recent):
    """A page to read (0 .. 2) or to write (3, 4), of one head: the whole row stays; the other is cut."""
    rows = [(3, 20), (4, 7)]
    cache, _ = _filled(rows, 4, 2, 64, 6, seed=2)
    cache["table"][0, 1, entry] = bad
    before, ref = _copy(cache), Mirror(cache)
    ref.t["table"][0, 1, entry] = _spare(before)
    ref.evict(2, recent)
    outs = {n + "_out": torch.full_like(cache[n], -5) for n in ("state", "table", "weight", "pos")} if apart else {}
    tra.paged_cache_evict(cache, keep=2, recent=recent, **outs)
    assert int(cache.status) == tra.DEV_BAD_CACHE
    _same_pages(cache, before, [p for p in range(cache.n_pool) if p not in before["table"][1, :, 4:].flatten().tolist()])
    for b, m in ((0, 3 * TILE + 20), (1, 2 * TILE + 7)):
        for n in ("state", "table", "weight", "pos"):
            got = (outs[n + "_out"] if apart else cache[n])[b].cpu().numpy()
            want = before[n][b].cpu().numpy() if b == 0 else ref.t[n][b]
            if n in ("weight", "pos"):
                got, want = got[:, :m], want[:, :m]
            assert np.array_equal(got, want), (b, n)
    for n in ("k8", "v8", "sk", "sv"):
        at = ref.t["table"][1, :, :2].flatten().tolist()
        assert np.array_equal(cache[n].cpu().numpy()[at], ref.t[n][at]), n
    if apart:
        for n in ("state", "table", "weight", "pos"):
            assert torch.equal(cache[n], before[n]), n


@pytest.mark.parametrize("cap", [5, 700])
@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
@pytest.mark.parametrize("head,entry,bad", [(1, 0, -1), (2, 2, 1 << 20), (0, 1, 2 ** 31 - 1), (1, 3, -2 ** 31)])
def test_step_keeps_a_row_with_a_bad_page(head, entry, bad, apart, cap):
    """Of three rows the middle one has a bad number in one head, the last one of a full tail's page among
    them: the row keeps its state, that head its output and weights, and put right it can be stepped."""
    rows, hkv, grp, d = [(2, 5), (3, 63), (1, 63)], 3, 2, 64
    cache, (q, kn, vn) = _filled(rows, hkv * grp, hkv, d, cap, seed=3)
    page = int(cache["table"][1, head, entry])
    cache["table"][1, head, entry] = bad
    out = _normal(_rng(1), 3, hkv * grp, d)
    first, before, ref = out.clone(), _copy(cache), Mirror(cache)
    ref.t["table"][1, head, entry] = page
    kw = dict(state_out=torch.full_like(cache["state"], 99), weight_out=torch.full_like(cache["weight"], 5.5)) if apart else {}
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1, **kw)
    assert int(cache.status) == tra.DEV_BAD_CACHE
    m = rows[1][0] * TILE + rows[1][1]
    state = kw.get("state_out", cache["state"])
    weight = kw.get("weight_out", cache["weight"])
    assert torch.equal(state[1], before["state"][1])
    assert torch.equal(weight[1, head, :m], before["weight"][1, head, :m])
    assert torch.equal(out[1, head * grp:(head + 1) * grp], first[1, head * grp:(head + 1) * grp])
    _same_pages(cache, before, before["table"][1, :, :3].flatten().tolist())
    assert torch.equal(cache["k_tail"][1, :, :63], before["k_tail"][1, :, :63])
    o, bound = ref.step(q, kn, vn, 0.1)
    ref.check_step(out, {key: x for key, x in o.items() if key != (1, head)}, bound, weight)
    assert state[0].tolist() == ref.t["state"][0].tolist() and state[2].tolist() == ref.t["state"][2].tolist()
    # put right, from the same start
    for n, x in before.items():
        cache[n].copy_(x)
    cache["table"][1, head, entry] = page
    cache.status.zero_()
    ref = Mirror(cache)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1)
    assert int(cache.status) == 0
    o, bound = ref.step(q, kn, vn, 0.1)
    ref.check_step(out, o, bound)
    ref.same()


@pytest.mark.parametrize("pages", [(147, 73, 36, 295, 0, 1), (147,) * 6, (295, 295, 295, 295)], ids=str)
def test_step_with_a_bad_page_in_a_long_list(pages):
    """Rows of one and of several CTAs, which end within a CTA's share of the list and (the equal ones: 4, 6
    and 8 items a CTA) with it: a bad number is found wherever it stands, and only there; the workspace's old
    contents count for nothing."""
    rows = [(n, 63) for n in pages]
    cache, (q, kn, vn) = _filled(rows, 4, 2, 64, 300, seed=4)
    good = cache["table"].clone()
    state = cache["state"].clone()
    out = torch.empty_like(q)
    at = [(r, g, i) for r, n in enumerate(pages) for g in (0, 1) for i in {0, n // 2, n}]
    for b, g, i in at:
        cache["table"].copy_(good)
        cache["state"].copy_(state)
        cache["table"][b, g, i] = -3
        cache.workspace.fill_(0xFF)
        cache.status.zero_()
        tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1)
        assert int(cache.status) == tra.DEV_BAD_CACHE
        for r, (n, _) in enumerate(rows):
            want = state[r, :2].tolist() if r == b else [n + 1, 0]
            assert cache["state"][r, :2].tolist() == want, (b, r)
