"""The evicting cache's calls as a program makes them: on streams of its own, captured, beside other
calls, and with states and pages that are not in order."""
import math

import numpy as np
import pytest
import torch

import tile_routed_mixed_causal_b200 as tra
from tile_routed_mixed_causal_b200 import api

from test_gpu_evicting import DEV, TILE, Mirror, _cu, _filled, _normal, _rng, _sums64

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


def test_importance_of_a_side_stream_on_the_current_one():
    """Prompt after prompt on a side stream, each result read on the current stream, late, and dropped: the
    next one is not written over it."""
    hq, hkv, d, n = 4, 2, 64, 500
    gen = _rng(22)
    q = [_normal(gen, n, hq, d) for _ in range(4)]
    k, shape, s = _normal(gen, n, hkv, d), tra.Shape([0, n], hq, hkv, d), torch.cuda.Stream()
    want = [api.prompt_importance(shape, x, k) for x in q]
    torch.cuda.synchronize()
    got = []
    for x in q:
        w = api.prompt_importance(shape, x, k, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(10_000_000)
        got.append(w.clone())
        del w
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


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


# ================================================================ which rows are cut
@pytest.mark.parametrize("least,cut", [(0, (0, 1, 3)), (4 * TILE + 63, (1, 3)), (4 * TILE + 64, (3,)), (2 ** 31 - 1, ())])
@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
def test_evict_from(least, cut, apart):
    """Rows below `least` tokens stay, whatever they hold."""
    rows = [(4, 62), (4, 63), (2, 63), (5, 0), (-1, 3)]
    cache, _ = _filled(rows, 4, 2, 64, 8, seed=7)
    before, ref = _copy(cache), Mirror(cache)
    for b in range(len(rows)):      # to the mirror, the others are idle
        if b not in cut:
            ref.t["state"][b, 0] = -1
    ref.evict(2, 30)
    for b in range(len(rows)):
        if b not in cut:
            ref.t["state"][b, 0] = rows[b][0]
    outs = {n + "_out": torch.full_like(cache[n], -5) for n in ("state", "table", "weight", "pos")} if apart else {}
    tra.paged_cache_evict(cache, keep=2, recent=30, least=least, **outs)
    assert int(cache.status) == 0
    if not apart:
        ref.same()
        return
    assert all(torch.equal(cache[n], before[n]) for n in ("state", "table", "weight", "pos", "k_tail", "v_tail"))
    ref.same("k8", "v8", "sk", "sv")
    assert np.array_equal(outs["state_out"].cpu().numpy(), ref.t["state"])
    assert np.array_equal(outs["table_out"].cpu().numpy(), ref.t["table"])
    for b in range(4):
        m = ref.t["state"][b, 0] * TILE + rows[b][1]
        for n in ("weight", "pos"):
            assert np.array_equal(outs[n + "_out"][b, :, :m].cpu().numpy(), ref.t[n][b, :, :m]), (b, n)


def _plan_steps(lens, which, seed, n, **kw):
    """A plan over the sequences `which` of a batch, n steps; per sequence its outputs, positions and
    weights after each step in which a row was cut, and the pages that every row had at every step."""
    hq, hkv, d = 4, 2, 64
    parts = []
    for i, T in enumerate(lens):
        gen = _rng(seed + i)
        parts.append([_normal(gen, T, h, d) for h in (hq, hkv, hkv)] + [[_normal(gen, n, h, d) for h in (hq, hkv, hkv)]])
    q, k, v = (torch.cat([parts[i][x] for i in which]) for x in range(3))
    shape = tra.Shape(_cu([lens[i] for i in which]), hq, hkv, d)
    plan = api.EvictingDecodePlan(shape, keep=2, limit=4, recent=70, **kw)
    plan.prefill(q, k, v)
    outs, pages = [], []
    for s in range(n):
        x = [torch.stack([parts[i][3][y][s] for i in which]) for y in range(3)]
        out = torch.empty_like(x[0])
        plan.step(*x, out)
        outs.append(out)
        pages.append([r[0] for r in plan.rows])
        assert plan.cache["state"][:, :2].cpu().tolist() == plan.rows
    assert int(plan.status) == 0
    return plan, torch.stack(outs), pages


def test_a_row_is_cut_alike_alone_and_beside_others():
    """With per_row a row's cuts, and so the tokens that it holds, are its own; without, the longest
    row's cuts are everybody's.  (Outputs: the batch changes how a row is split, its fp32 sums' order and a
    bf16 rounding, 2^-8 of values up to 4.)"""
    lens, n = [300, 130, 64], 330
    plan, outs, pages = _plan_steps(lens, (0, 1, 2), 40, n, per_row=True)
    cuts = [[s for s in range(1, n) if pages[s][b] < pages[s - 1][b]] for b in range(3)]
    assert all(cuts) and cuts[0] != cuts[1] != cuts[2]
    for b in range(3):
        alone, o, p = _plan_steps(lens, (b,), 40, n, per_row=True)
        assert [x[0] for x in p] == [x[b] for x in pages]
        m = pages[-1][b] * TILE + plan.rows[b][1]
        assert torch.equal(alone.cache["pos"][0, :, :m], plan.cache["pos"][b, :, :m])
        assert float((alone.cache["weight"][0, :, :m] - plan.cache["weight"][b, :, :m]).abs().max()) < 1e-3
        assert float((o[:, 0].float() - outs[:, b].float()).abs().max()) <= 2.0 ** -6
    _, _, pages = _plan_steps(lens, (0, 1, 2), 40, n)
    cuts = [[s for s in range(1, n) if pages[s][b] < pages[s - 1][b]] for b in range(3)]
    assert cuts[0][0] in cuts[1] and cuts[0][0] in cuts[2]


def test_retired_row():
    """A row that is done keeps what it holds, gets no output and causes no cut of the others."""
    hq, hkv, d, lens = 4, 2, 64, [190, 64]
    gen, cu = _rng(51), _cu(lens)
    q, k, v = (_normal(gen, cu[-1], h, d) for h in (hq, hkv, hkv))
    plan = api.EvictingDecodePlan(tra.Shape(cu, hq, hkv, d), keep=1, limit=2, recent=10)
    plan.prefill(q, k, v)
    plan.retire(0)
    held = _copy(plan.cache)
    for i in range(80):
        x = [_normal(gen, 2, h, d) for h in (hq, hkv, hkv)]
        out = torch.full_like(x[0], 5.0)
        plan.step(*x, out)
        assert bool((out[0] == 5.0).all()) and not bool((out[1] == 5.0).any())
        assert plan.rows == [[-1, 62], [1 + (i + 1) // TILE, (i + 1) % TILE]]
        assert plan.cache["state"][:, :2].cpu().tolist() == plan.rows
    for n in ("state", "table", "weight", "pos", "k_tail", "v_tail"):
        assert torch.equal(plan.cache[n][0], held[n][0]), n
    plan.prefill(q, k, v)
    assert plan.cache["state"][:, :2].cpu().tolist() == plan.rows == [[1, 62], [1, 0]]


def test_captured_cut_and_step():
    """What a plan does, captured from the calls themselves: the rows' states decide at every replay."""
    lens, n = [300, 130], 300
    hq, hkv, d = 4, 2, 64
    gen, cu = _rng(61), _cu(lens)
    q, k, v = (_normal(gen, cu[-1], h, d) for h in (hq, hkv, hkv))
    x = [_normal(gen, 2, h, d) for h in (hq, hkv, hkv)]
    shape = tra.Shape(cu, hq, hkv, d)
    plans = [api.EvictingDecodePlan(shape, keep=2, limit=4, recent=70, per_row=True) for _ in range(2)]
    outs = [torch.empty_like(x[0]) for _ in plans]
    for p in plans:
        p.prefill(q, k, v)
    tra.paged_cache_evict(plans[0].cache, keep=4, least=2 ** 30)     # loads the kernels, cuts nothing
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        tra.paged_cache_evict(plans[0].cache, keep=2, recent=70, least=4 * TILE + 63)
        tra.paged_attention_decode(plans[0].cache, *x, outs[0], softmax_scale=0.125)
    for i in range(n):
        for y, z in zip(x, (hq, hkv, hkv)):
            y.copy_(_normal(_rng(100 + i), 2, z, d))
        g.replay()
        plans[1].step(*x, outs[1], scale=0.125)
        assert torch.equal(*outs), i
    for name in plans[0].cache.NAMES:
        assert torch.equal(plans[0].cache[name], plans[1].cache[name]), name
    assert int(plans[0].status) == 0


# ================================================================ sums over a given lse
def _scores_of(kind, gen, T, h, d):
    x = torch.randn(T, h, d, generator=gen, device=DEV)
    if kind == "whole":         # small whole numbers: every score is exact in fp32
        return torch.randint(0, 5, (T, h, d), generator=gen, device=DEV).to(torch.bfloat16)
    if kind == "positive":
        x = x.abs() * 2
    if kind == "outliers":
        x[..., 5:9] *= 10
    if kind == "large":
        x *= 2.8
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("own", [False, True], ids=["lse in 64 bits", "lse of the call"])
@pytest.mark.parametrize("kind", ["whole", "positive", "outliers", "large", "small"])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_a_given_lse_have_no_bias(d, kind, own):
    """All weights together against the definition with that lse, at scores up to 200: whatever the tensor
    core cuts off must not depend on what the values are like, nor on where the lse comes from.

    Bound of the mean: n = d / 16 MMAs cut a partial sum P_k - f L, L = lse / scale, off by half of its
    last place in the mean, 0.36 * 2^-23 of it (its mantissa spread evenly over a factor of two).  With
    f = (n + 1) / 2n these add up to nothing for a score S = L; for S < L they leave (n + 1) / 2 times
    L - S, whose mean is the row's entropy, at most log T.  What partial sums that do not grow evenly
    leave is taken as a quarter of all that is cut off, sum_k |k / n - f| times 2^-24 L.  Exponents and
    sums: 2^-20.  (Without a start value it is 0.36 (n + 1) / 2 * 2^-23 L: 2e-7 L at d = 128.)"""
    T, hq, hkv, n = 3000, 4, 2, d // 16
    gen, scale = _rng(d), 1.0 / math.sqrt(d)
    q, k = _scores_of(kind, gen, T, hq, d), _scores_of(kind, gen, T, hkv, d)
    shape = tra.Shape([0, T], hq, hkv, d)
    w, lse = torch.empty(T, hkv, device=DEV), torch.empty(hq, T, device=DEV)
    if own:
        tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=scale)
    else:
        lse.copy_(_sums64(q, k, [0, T], 0, scale)[1])
    ref = _sums64(q, k, [0, T], 0, scale, lse)[0]
    tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=scale, lse_given=True)
    f = (n + 1) / (2 * n)
    top = float(lse.abs().max())
    uneven = 0.25 * sum(abs(i / n - f) for i in range(1, n + 1)) * 2.0 ** -24 * top
    bound = 0.36 * 2.0 ** -23 * (n + 1) / 2 * math.log(T) + uneven + 2.0 ** -20
    assert abs(float(w.double().sum() / ref.sum()) - 1.0) < bound
    rel = 2.0 ** -22 * 2 * top * 1.4427 + 2.0 ** -18      # of one weight: every cut-off to one side
    assert bool(((w.double() - ref).abs() <= rel * ref + 1e-30).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 1e6, 1e30])
def test_sums_over_a_given_lse_at_far_scales(scale):
    """Scales at the ends of the range, scores of ordinary size times the scale, and an lse far from
    the scores: zeroes where the definition has them."""
    T, hq, hkv, d = 200, 2, 1, 64
    gen = _rng(3)
    root = math.sqrt(1.0 / (scale * math.sqrt(d)))
    q = (torch.randn(T, hq, d, generator=gen, device=DEV) * root).to(torch.bfloat16)
    k = (torch.randn(T, hkv, d, generator=gen, device=DEV) * root).to(torch.bfloat16)
    shape = tra.Shape([0, T], hq, hkv, d)
    w = torch.empty(T, hkv, device=DEV)
    for shift in (0.0, 1e4, 1e30, 3e38):
        lse = (_sums64(q, k, [0, T], 0, scale)[1] + shift).float()
        ref = _sums64(q, k, [0, T], 0, scale, lse)[0]
        tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=scale, lse_given=True)
        assert bool(((w.double() - ref).abs() <= 2.0 ** -17 * ref + 1e-30).all()), shift


@pytest.mark.parametrize("T", [200, 3000])
def test_infinite_sums(T):
    """An lse far below the scores: sums past fp32's range are infinite, not NaN, key by key."""
    hq, hkv, d = 2, 1, 64
    gen = _rng(4)
    q, k = _normal(gen, T, hq, d), _normal(gen, T, hkv, d)
    shape = tra.Shape([0, T], hq, hkv, d)
    lse = _sums64(q, k, [0, T], 0, 0.125)[1].float()
    w = torch.empty(T, hkv, device=DEV)
    lse[0, T // 2] = -1e5           # one query: the keys up to it are seen by it
    ref = _sums64(q, k, [0, T], 0, 0.125, lse)[0]
    assert bool(torch.isinf(ref[:T // 2 + 1]).all()) and bool(torch.isfinite(ref[T // 2 + 1:]).all())
    tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=0.125, lse_given=True)
    assert bool((w[:T // 2 + 1] == math.inf).all())
    assert bool(((w.double() - ref)[T // 2 + 1:].abs() <= 2.0 ** -17 * ref[T // 2 + 1:]).all())
    lse -= 1e5
    tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=0.125, lse_given=True)
    assert bool((w == math.inf).all())


# ================================================================ probabilities against V
@pytest.mark.parametrize("cap", [5, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_values_that_cancel(d, cap):
    """Eight tokens of a row have values, of either sign: where they cancel, what P is rounded to shows past the
    output's own rounding.  Bounds: the output's bf16, half a step 2^-8; of the sum of p |v|: exponents (|q| |k|
    in fp32, 2 * 2^-22 of it, as for every score), ex2 and sums 2^-18, P in two f16 parts 2^-21."""
    B, grp = 64, 8
    cache, (q, kn, vn) = _filled([(1, 0)] * B, grp, 1, d, cap, seed=9)
    cache["sk"].fill_(1.0 / 64)
    cache["sv"].fill_(1.0 / 64)
    cache["v8"][:, 8:] = 0
    vn.zero_()
    pages = cache["table"][:, 0, 0].long()
    k = torch.cat([cache["k8"][pages].double() / 64, kn.double()], 1)
    v = torch.cat([cache["v8"][pages].double() / 64, vn.double()], 1)
    scale = 1.0 / math.sqrt(d)
    p = torch.softmax(q.double() @ k.mT * scale, -1)
    o, mag = p @ v, p @ v.abs()
    assert int((o.abs() < 0.002 * mag).sum()) > 20
    out = torch.empty_like(q)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=scale)
    size = float((q.double().abs() @ k.abs().mT).max()) * scale * 1.4427
    rel = 2 * size * 2.0 ** -22 * math.log(2) + 2.0 ** -18 + 2.0 ** -21
    assert bool(((out.double() - o).abs() <= 2.0 ** -8 * o.abs() + rel * mag).all())
