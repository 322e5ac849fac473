"""GPU parity of the weight sums and the evicting key / value cache against plain 64-bit
implementations.  What is held in whole numbers (codes, positions, states, page tables) and
what is only moved (weights of survivors, tails) has to be equal; the rest is bounded by the
roundings of the path, stated at each bound.
"""
import math

import numpy as np
import pytest
import torch

import tile_routed_mixed_causal_b200 as tra
from tile_routed_mixed_causal_b200 import api

pytestmark = pytest.mark.gpu
TILE = 64
DEV = "cuda"


def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape, outliers=False):
    x = torch.randn(shape, generator=gen, device=DEV)
    if outliers:
        x[..., :2] *= 10.0
    return x.to(torch.bfloat16)


def _cu(lens):
    return [0] + np.cumsum(lens).tolist()


# ================================================================ weight sums
def _sums64(q, k, cu, n_queries, scale, lse=None):
    """(weights, lse, exponent size): from the definition, in 64 bits.  The last: per query
    row, |scale| sum_c |q_c| |k_c| at its largest, in log2 units."""
    hq, hkv = q.shape[1], k.shape[1]
    grp = hq // hkv
    w = torch.zeros(k.shape[0], hkv, dtype=torch.float64, device=DEV)
    z = torch.zeros(hq, q.shape[0], dtype=torch.float64, device=DEV)
    size = 0.0
    for t0, t1 in zip(cu, cu[1:]):
        T = t1 - t0
        if T == 0:
            continue
        W = min(T, n_queries) if n_queries else T
        i = torch.arange(T - W, T, device=DEV)
        see = torch.arange(T, device=DEV)[None, :] <= i[:, None]
        for h in range(hq):
            qq, kk = q[t1 - W:t1, h].double(), k[t0:t1, h // grp].double()
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            if lse is None:
                row = torch.logsumexp(s, 1)
            else:
                row = lse[h, t1 - W:t1].double()
            z[h, t1 - W:t1] = row
            p = torch.exp(s - row[:, None])
            p[~torch.isfinite(row)] = 0.0
            w[t0:t1, h // grp] += p.sum(0)
            size = max(size, float((qq.abs() @ kk.abs().T).max()) * scale * 1.4427)
    return w, z, size


def _weight_bounds(size, lse):
    """Relative bound of a weight and absolute bound of an lse.  Scores: fp32 sums of exact
    products, at most d roundings of which those of the tensor core may truncate: 2^-22 of the sum of
    magnitudes (size) covers d = 128 of random sign (each 2^-23 of a partial sum); the scale's
    rounding, the lse's own, its product with log2(e) and the fused subtraction: 4 * 2^-24 of the
    exponents.  ex2: 2^-21; the sums: 64 columns in fp32, then compensated: 2^-18 in all."""
    top = float(torch.nan_to_num(lse, nan=0.0, posinf=0.0, neginf=0.0).abs().max()) * 1.4427
    delta = (size + top) * 2.0 ** -22
    return delta * math.log(2) + 2.0 ** -18, delta * math.log(2) + 2.0 ** -18 + top * 2.0 ** -23


SUM_CASES = [
    # heads, d, lengths, window
    (4, 2, 128, [1], 0), (4, 2, 64, [2, 1, 0, 3], 0), (2, 2, 64, [63, 64, 65], 0), (8, 2, 128, [127, 128, 129], 0),
    (7, 1, 128, [300, 5], 0), (8, 1, 64, [700], 0), (4, 4, 128, [257, 0, 640], 0),
    (8, 2, 128, [1000], 1), (8, 2, 64, [130, 7, 64], 1), (32, 8, 128, [700, 64, 65], 64), (8, 1, 128, [900], 16),
    (14, 2, 64, [513], 33), (6, 2, 128, [40, 300, 129], 40), (2, 2, 128, [600], 128), (4, 2, 64, [600, 90], 200),
    (12, 4, 128, [333], 500), (16, 2, 128, [1, 64, 2], 5), (8, 1, 64, [60, 17], 0),
]


# prompts of very different lengths
SUM_RAGGED = [(4, 2, 64, [0, 1500, 3, 0, 90, 64, 1, 200, 0], 0), (8, 2, 128, [5] * 40 + [900] + [130, 1] * 9, 0),
              (8, 2, 128, [1] * 33 + [1200, 0, 700], 64), (2, 1, 64, [10, 0, 2000], 300)]
# many heads to a KV head: a query tile of few tokens
SUM_GROUPS = [(32, 1, 64, [77, 3], 2), (64, 2, 128, [40], 1), (128, 1, 64, [9, 200], 1), (96, 1, 128, [70], 3), (24, 1, 64, [130], 9)]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("hq,hkv,d,lens,window", SUM_CASES + SUM_GROUPS + SUM_RAGGED, ids=str)
def test_weight_sums(hq, hkv, d, lens, window, given):
    gen = _rng(len(lens) + 7 * window + d)
    cu = _cu(lens)
    q, k = _normal(gen, cu[-1], hq, d), _normal(gen, cu[-1], hkv, d)
    scale = 1.0 / math.sqrt(d)
    shape = tra.Shape(cu, hq, hkv, d)
    lse = torch.full((hq, cu[-1]), 7.25, device=DEV)
    ref_in = None
    if given:
        lse.copy_(_sums64(q, k, cu, window, scale)[1])
        ref_in = lse.clone()
    before = lse.clone()
    w = torch.full((cu[-1], hkv), math.nan, device=DEV)
    tra.attention_weight_sums(shape, q, k, w, lse, n_queries=window, softmax_scale=scale, lse_given=given)
    assert int(shape.status) == 0
    ref, z, size = _sums64(q, k, cu, window, scale, ref_in)
    rel, ab = _weight_bounds(size, z)
    assert bool((w.double() - ref).abs().le(rel * ref + 1e-30).all())
    inside = torch.zeros(cu[-1], dtype=torch.bool, device=DEV)
    for t0, t1 in zip(cu, cu[1:]):
        inside[t1 - (min(t1 - t0, window) if window else t1 - t0):t1] = True
    if given:
        assert torch.equal(lse, before)
    else:
        assert bool((lse.double() - z)[:, inside].abs().le(ab).all())
        assert torch.equal(lse[:, ~inside], before[:, ~inside])
    # the sums run in a fixed order
    w2, l2 = torch.empty_like(w), before.clone()
    tra.attention_weight_sums(shape, q, k, w2, l2, n_queries=window, softmax_scale=scale, lse_given=given)
    assert torch.equal(w, w2) and torch.equal(lse, l2)


@pytest.mark.parametrize("hq,hkv,d,T,window", [(2, 1, 64, 5000, 0), (8, 2, 128, 4096, 64), (4, 4, 128, 2600, 0)])
def test_weight_sums_long(hq, hkv, d, T, window):
    """Few units with long streams: CTAs share a unit and join their sums."""
    gen = _rng(T)
    q, k = _normal(gen, T, hq, d, outliers=True), _normal(gen, T, hkv, d, outliers=True)
    scale = 1.0 / math.sqrt(d)
    shape = tra.Shape([0, T], hq, hkv, d)
    w, lse = torch.zeros(T, hkv, device=DEV), torch.zeros(hq, T, device=DEV)
    tra.attention_weight_sums(shape, q, k, w, lse, n_queries=window, softmax_scale=scale)
    ref, z, size = _sums64(q, k, [0, T], window, scale)
    rel, ab = _weight_bounds(size, z)
    assert bool((w.double() - ref).abs().le(rel * ref + 1e-30).all())
    assert bool((lse.double() - z)[:, T - (window or T):].abs().le(ab).all())
    # the probabilities of a query sum to one: so do the weights over all keys
    assert float(w.double().sum()) == pytest.approx((window or T) * hq, rel=rel)


def test_weight_sums_ignore_what_is_masked():
    """Rows whose lse is not finite add nothing, and nothing of another sequence or of a later key
    reaches a sum, whatever it is."""
    hq, hkv, d, lens = 4, 2, 128, [100, 70, 129]
    gen, cu = _rng(3), _cu(lens)
    q, k = _normal(gen, cu[-1], hq, d), _normal(gen, cu[-1], hkv, d)
    shape, scale = tra.Shape(cu, hq, hkv, d), 1.0 / math.sqrt(d)
    lse = _sums64(q, k, cu, 0, scale)[1].float()
    lse[1, 20] = math.inf
    lse[2, 30:40] = -math.inf
    lse[3, 299 - 1] = math.nan
    ref = _sums64(q, k, cu, 0, scale, lse)[0]
    w = torch.empty(cu[-1], hkv, device=DEV)
    tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=scale, lse_given=True)
    rel = _weight_bounds(40.0, lse)[0]
    assert bool((w.double() - ref).abs().le(rel * ref + 1e-30).all())
    # a NaN sequence in the middle
    q[100:170], k[100:170] = math.nan, math.inf
    w2, l2 = torch.empty_like(w), torch.empty_like(lse)
    tra.attention_weight_sums(shape, q, k, w2, l2, softmax_scale=scale)
    assert bool(torch.isfinite(w2[:100]).all()) and bool(torch.isfinite(w2[170:]).all())
    assert bool(torch.isfinite(l2[:, :100]).all()) and bool(torch.isfinite(l2[:, 170:]).all())


def test_prompt_importance_selects_for_the_hybrid():
    """The sums as hybrid_select_tokens' importance, from the lse of a prefill."""
    hq, hkv, d, lens = 8, 2, 128, [500, 130]
    gen, cu = _rng(5), _cu(lens)
    q, k, v = (_normal(gen, cu[-1], h, d) for h in (hq, hkv, hkv))
    shape = tra.Shape(cu, hq, hkv, d)
    plan = api.PrefillPlan(shape, tra.Policy.boundary([8] * hq, [8] * hq))
    out, lse = torch.zeros_like(q), torch.zeros(hq, cu[-1], device=DEV)
    plan.run(q, k, v, out, lse)
    w = api.prompt_importance(shape, q, k, n_queries=64, lse=lse)
    dense = api.prompt_importance(shape, q, k, n_queries=64)
    # the prefill's scores come from INT8 codes: its weights are near those of the dense rows
    assert float((w - dense).abs().max()) < 0.1 * float(dense.max())
    hy = tra.Hybrid(shape, 0.1, 16)
    tra.hybrid_select_tokens(shape, w, 0.1, k, v, hy)
    for b, (t0, t1) in enumerate(zip(cu, cu[1:])):
        n = math.ceil(0.1 * (t1 - t0))
        for g in range(hkv):
            x = w[t0:t1, g].cpu().numpy()
            want = np.sort(np.lexsort((np.arange(len(x)), -x))[:n])
            assert hy.sel_pos[b, g, :n].cpu().tolist() == want.tolist()


# ================================================================ the cache, in 64 bits
def _quant(x):
    """Codes and scale of a block (float32 values): by the definition, with numpy's IEEE fp32."""
    x = np.asarray(x, np.float32)
    s = np.float32(np.max(np.abs(x))) / np.float32(127.0)
    if s == 0:
        return np.zeros(x.shape, np.int8), s
    return np.clip(np.rint(x / s), -127, 127).astype(np.int8), s


def _pick(weight, first, count):
    """The count tokens from `first` on, then of largest weight, ties to the earlier; ascending."""
    j = np.arange(len(weight))
    w = np.asarray(weight, np.float64)
    return np.sort(np.lexsort((j, -w, j < first))[:count])


class Mirror:
    """The cache's arrays on the host, changed by the definitions."""

    def __init__(self, cache):
        self.c = cache
        self.pull()

    def pull(self):
        self.t = {n: (x.float() if x.dtype == torch.bfloat16 else x).cpu().numpy().copy() for n, x in self.c.t.items()}

    def same(self, *names):
        for n in names or self.c.NAMES:
            x = self.c[n]
            got = (x.float() if x.dtype == torch.bfloat16 else x).cpu().numpy()
            assert np.array_equal(got, self.t[n]), n

    def fill(self, cu, k, v, weights, keep, recent):
        t = self.t
        k, v = k.float().cpu().numpy(), v.float().cpu().numpy()
        w = None if weights is None else weights.cpu().numpy()
        for b, (t0, t1) in enumerate(zip(cu, cu[1:])):
            T = t1 - t0
            body = T // TILE * TILE
            n = min(body // TILE, keep)
            m, tail = n * TILE, T - body
            t["state"][b] = (n, tail, T, 0)
            for g in range(self.c.Hkv):
                wg = np.zeros(T, np.float32) if w is None else w[t0:t1, g]
                first = body - m if w is None else max(T - recent, body - m)
                at = np.concatenate([_pick(wg[:body], first, m), np.arange(body, T)]).astype(np.int64)
                t["weight"][b, g, :m + tail] = wg[at]
                t["pos"][b, g, :m + tail] = at
                for x, code, sc, tl in ((k, "k8", "sk", "k_tail"), (v, "v8", "sv", "v_tail")):
                    rows = x[t0:t1, g][at]
                    t[tl][b, g, :tail] = rows[m:]
                    for i in range(n):
                        page = t["table"][b, g, i]
                        t[code][page], t[sc][page] = _quant(rows[i * TILE:(i + 1) * TILE])

    def evict(self, keep, recent):
        t = self.t
        for b in range(self.c.B):
            n, tail = t["state"][b, :2]
            if n <= keep or n + keep > self.c.cap:
                continue
            body, m = n * TILE, keep * TILE
            for g in range(self.c.Hkv):
                tab = t["table"][b, g].copy()
                at = _pick(t["weight"][b, g, :body], max(body + tail - recent, body - m), m)
                at = np.concatenate([at, np.arange(body, body + tail)])
                for name in ("weight", "pos"):
                    t[name][b, g, :m + tail] = t[name][b, g][at].copy()
                for code, sc in (("k8", "sk"), ("v8", "sv")):
                    src = tab[at[:m] // TILE]
                    x = t[code][src, at[:m] % TILE].astype(np.float32) * t[sc][src][:, None]
                    for i in range(keep):
                        page = tab[n + i]
                        t[code][page], t[sc][page] = _quant(x[i * TILE:(i + 1) * TILE])
                t["table"][b, g] = np.concatenate([tab[n:n + keep], tab[:n], tab[n + keep:]])
            t["state"][b, 0] = keep

    def step(self, q, k_new, v_new, scale):
        """Outputs, their bounds, the new weights and their bounds; what is exact goes into the mirror."""
        t, c = self.t, self.c
        grp = c.Hq // c.Hkv
        q, k_new, v_new = (x.double().cpu().numpy() for x in (q, k_new, v_new))
        out, bound = {}, {}
        for b in range(c.B):
            n, tl, seen = t["state"][b, :3]
            if n < 0 or (tl == TILE - 1 and n == c.cap):
                continue
            m = n * TILE + tl
            for g in range(c.Hkv):
                t["k_tail"][b, g, tl], t["v_tail"][b, g, tl] = k_new[b, g], v_new[b, g]
                t["pos"][b, g, m] = seen
                pg = t["table"][b, g, :n]
                rows = [np.concatenate([(t[cd][pg].astype(np.float64) * t[sc][pg].astype(np.float64)[:, None, None]).reshape(-1, c.d),
                                        t[tt][b, g, :tl + 1].astype(np.float64)])
                        for cd, sc, tt in (("k8", "sk", "k_tail"), ("v8", "sv", "v_tail"))]
                qq = q[b, g * grp:(g + 1) * grp]
                s = qq @ rows[0].T * scale
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                # exponents as in _weight_bounds
                size = (np.abs(qq) @ np.abs(rows[0]).T).max() * scale * 1.4427
                rel = 2 * size * 2.0 ** -22 * math.log(2) + 2.0 ** -18
                # P in f16 (half a step 2^-11, 2^-25 below its normal range, against a sum of at least
                # one), the output in bf16 (2^-8)
                vmax = np.abs(rows[1]).max()
                o = p @ rows[1]
                out[b, g] = o
                bound[b, g] = (2.0 ** -8 * np.abs(o) + (2.0 ** -10.9 + rel) * (p @ np.abs(rows[1])) +
                               len(s[0]) * 2.0 ** -25 * vmax)
                old = t["weight"][b, g, :m + 1].copy()
                old[m] = 0.0
                t["weight"][b, g, :m + 1] = (old.astype(np.float64) + p.sum(0)).astype(np.float32)
                # (a head's probability below the smallest normal number, 2^-126, counts as zero: ex2
                # flushes it, which is off by less than that number)
                bound["w", b, g] = rel * p.sum(0) + 2.0 ** -22 * t["weight"][b, g, :m + 1] + grp * 2.0 ** -126
            if tl == TILE - 1:
                for g in range(c.Hkv):
                    page = t["table"][b, g, n]
                    for cd, sc, tt in (("k8", "sk", "k_tail"), ("v8", "sv", "v_tail")):
                        t[cd][page], t[sc][page] = _quant(t[tt][b, g])
            t["state"][b] = (n + (tl == TILE - 1), (tl + 1) % TILE, seen + 1, t["state"][b, 3])
        return out, bound

    def check_step(self, got, out, bound, weight=None, before=None):
        """got: the call's output, weight: where its weights went (default: the cache's own)."""
        grp = self.c.Hq // self.c.Hkv
        got = got.double().cpu().numpy()
        w = (self.c["weight"] if weight is None else weight).cpu().numpy()
        for key, o in out.items():
            b, g = key
            assert np.all(np.abs(got[b, g * grp:(g + 1) * grp] - o) <= bound[key]), key
            m = len(bound["w", b, g])
            assert np.all(np.abs(w[b, g, :m].astype(np.float64) - self.t["weight"][b, g, :m]) <= bound["w", b, g]), key
            self.t["weight"][b, g, :m] = w[b, g, :m]    # go on from the kernel's own
        if before is not None:      # rows that take no part keep their output
            for b in range(self.c.B):
                if (b, 0) not in out:
                    assert np.array_equal(got[b], before[b]), b


def _filled(rows, hq, hkv, d, cap, seed, extra=3, v_scale=1.0, q_scale=1.0, ties=False):
    """A cache with rows of (pages, tail), random contents everywhere (so that nothing reads what is
    not there unnoticed), shuffled pages; and a step's inputs."""
    gen = _rng(seed)
    B = len(rows)
    n_pool = B * hkv * cap + extra
    z = lambda *s, t=torch.float32: torch.zeros(s, device=DEV, dtype=t)  # noqa: E731
    t = dict(k8=torch.randint(-127, 128, (n_pool, TILE, d), generator=gen, device=DEV, dtype=torch.int8),
             v8=torch.randint(-127, 128, (n_pool, TILE, d), generator=gen, device=DEV, dtype=torch.int8),
             sk=torch.rand(n_pool, generator=gen, device=DEV) * 0.02 + 0.005,
             sv=(torch.rand(n_pool, generator=gen, device=DEV) * 0.05 + 0.01) * v_scale,
             table=torch.randperm(n_pool, generator=gen, device=DEV)[:B * hkv * cap].to(torch.int32).view(B, hkv, cap),
             state=z(B, 4, t=torch.int32),
             weight=torch.rand(B, hkv, (cap + 1) * TILE, generator=gen, device=DEV) ** 4,
             pos=torch.cumsum(torch.randint(1, 3, (B, hkv, (cap + 1) * TILE), generator=gen, device=DEV), 2).to(torch.int32),
             k_tail=_normal(gen, B, hkv, TILE, d), v_tail=(_normal(gen, B, hkv, TILE, d) * v_scale).to(torch.bfloat16))
    if ties:
        t["weight"] = torch.round(t["weight"] * 6)      # a handful of values, most of them zero
        t["weight"][0, 0, 5] = -0.0
    for b, (n, tl) in enumerate(rows):
        t["state"][b] = torch.tensor([n, tl, max(0, n) * 2 * TILE + tl, 3 * b], dtype=torch.int32)
    cache = tra.PagedCache(B, hq, hkv, d, cap, tensors=t)
    step = ((_normal(gen, B, hq, d) * q_scale).to(torch.bfloat16), _normal(gen, B, hkv, d),
            (_normal(gen, B, hkv, d) * v_scale).to(torch.bfloat16))
    return cache, step


# ================================================================ fill
FILLS = [
    # heads, d, lengths, keep, recent
    (4, 2, 64, [0, 1, 63, 64], 2, 0), (8, 2, 128, [65, 128, 640], 3, 0), (8, 2, 128, [640, 1000], 3, 100),
    (2, 1, 64, [2000], 7, 5000), (4, 4, 128, [700, 10], 20, 10), (8, 1, 128, [4097], 16, 64),
    (4, 2, 64, [1500, 200, 64 * 9 + 63], 1, 70), (3, 3, 128, [9000], 64, 0),
]


@pytest.mark.parametrize("weights", ["random", "ties", None])
@pytest.mark.parametrize("hq,hkv,d,lens,keep,recent", FILLS, ids=str)
def test_fill(hq, hkv, d, lens, keep, recent, weights):
    gen, cu = _rng(keep + d), _cu(lens)
    k, v = _normal(gen, cu[-1], hkv, d, outliers=True), _normal(gen, cu[-1], hkv, d)
    w = None
    if weights:
        w = torch.randn(cu[-1], hkv, generator=gen, device=DEV)     # negative ones, too
        if weights == "ties":
            w = torch.round(w)
            w[w.abs() < 0.5] = 0.0
            w[::3][w[::3] == 0] = -0.0
    cache, _ = _filled([(2, 5)] * len(lens), hq, hkv, d, keep + 2, seed=keep)
    ref = Mirror(cache)
    shape = tra.Shape(cu, hq, hkv, d)
    tra.paged_cache_fill(cache, shape, k, v, keep=keep, recent=recent, weights=w)
    assert int(cache.status) == 0
    ref.fill(cu, k, v, w, keep, recent)
    ref.same()


def test_fill_of_many_tokens():
    """More tokens than the selection holds at a time."""
    T, gen = 64 * 1300 + 11, _rng(9)
    k, v = _normal(gen, T, 1, 64), _normal(gen, T, 1, 64)
    w = torch.round(torch.rand(T, 1, generator=gen, device=DEV) * 50)
    cache, _ = _filled([(-1, 0)], 2, 1, 64, 1000, seed=2)
    ref = Mirror(cache)
    tra.paged_cache_fill(cache, tra.Shape([0, T], 2, 1, 64), k, v, keep=900, recent=77, weights=w)
    ref.fill([0, T], k, v, w, 900, 77)
    ref.same()


def test_fill_values_at_the_borders():
    """Blocks of zeros, of the smallest and of huge values, of exact halves, of one outlier."""
    hkv, d, T = 2, 64, 64 * 8
    gen = _rng(4)
    k = _normal(gen, T, hkv, d)
    v = _normal(gen, T, hkv, d)
    k[0:64] = 0.0
    k[64:128] = (k[64:128].float() * 2.0 ** -125).to(torch.bfloat16)     # denormal quotients and scales
    k[128:192] = (k[128:192].float() * 1e36).to(torch.bfloat16)
    k[192:256] = torch.where(k[192:256] > 0, 2.0, -1.0).to(torch.bfloat16)  # every value is the largest or its half
    k[256:320, :, 0] = 1e30
    k[320:384] = torch.round(k[320:384].float() * 16).to(torch.bfloat16)
    k[320, :, 0] = 127.0 * 0.5                                            # a scale of 1/2: halves everywhere
    k[384:448] = 0.0
    k[384, 0, 5] = 2.0 ** -133                                            # the smallest bf16 alone
    cache, _ = _filled([(-1, 0)], hkv, hkv, d, 10, seed=6)
    ref = Mirror(cache)
    tra.paged_cache_fill(cache, tra.Shape([0, T], hkv, hkv, d), k, v, keep=8)
    ref.fill([0, T], k, v, None, 8, 0)
    ref.same()


@pytest.mark.parametrize("exponent", [0, 57, -60, -91, -92, -94, -110])
def test_fill_every_quotient(exponent):
    """Every quotient of a bf16 value and a largest value that does not round to zero: page i has the
    largest value (128 + i) 2^exponent and all X 2^-j below it, both signs."""
    x = torch.arange(128, 256, dtype=torch.float64)
    vals = torch.cat([x * 2.0 ** -j for j in range(11)])
    pages = []
    for a in range(128, 256):
        v = vals[vals <= a]
        v = torch.cat([v, -v, torch.tensor([float(a)])])
        pages.append(torch.cat([v, torch.zeros(TILE * 64 - len(v), dtype=torch.float64)]).view(TILE, 64))
    k = (torch.cat(pages) * 2.0 ** exponent).to(torch.bfloat16)
    assert torch.equal(k.double(), torch.cat(pages) * 2.0 ** exponent)
    k = k.to(DEV)[:, None].contiguous()
    T = k.shape[0]
    cache, _ = _filled([(-1, 0)], 1, 1, 64, 128, seed=6)
    ref = Mirror(cache)
    tra.paged_cache_fill(cache, tra.Shape([0, T], 1, 1, 64), k, -k, keep=128)
    ref.fill([0, T], k, -k, None, 128, 0)
    ref.same()


# ================================================================ decode
STEPS = [
    # heads, d, cap, rows (pages, tail)
    (4, 2, 128, 3, [(0, 0)]), (8, 1, 64, 3, [(1, 0), (0, 1), (0, 62)]), (32, 8, 128, 9, [(8, 17)]),
    (7, 1, 128, 6, [(5, 63), (-1, 0), (6, 62), (3, 0)]), (8, 8, 64, 5, [(4, 30), (5, 63), (2, 15), (-7, 9)]),
    (12, 4, 64, 40, [(37, 16), (1, 31), (39, 48)]), (16, 2, 128, 33, [(33, 3), (20, 63)]), (2, 2, 128, 70, [(64, 1)]),
    (6, 2, 128, 12, [(11, 47), (0, 63), (5, 32), (2, 33)] * 3), (8, 8, 128, 130, [(128, 40), (70, 63)]),
    # room for many pages: a warp takes whole pages
    (32, 8, 128, 300, [(8, 17)]), (14, 2, 64, 600, [(37, 16), (20, 63)]), (8, 8, 128, 400, [(128, 40), (70, 63)]),
    (7, 1, 128, 1300, [(300, 62), (-1, 0), (5, 63)]), (2, 1, 64, 1300, [(900, 5), (0, 0)]),
]


@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
@pytest.mark.parametrize("hq,hkv,d,cap,rows", STEPS, ids=str)
def test_decode(hq, hkv, d, cap, rows, apart):
    cache, (q, kn, vn) = _filled(rows, hq, hkv, d, cap, seed=cap + d)
    ref = Mirror(cache)
    scale = 1.0 / math.sqrt(d)
    out = _normal(_rng(1), len(rows), hq, d)
    before = out.double().cpu().numpy()
    kw, own = {}, {n: cache[n].clone() for n in ("state", "weight")}
    if apart:
        kw = dict(state_out=torch.full_like(cache["state"], 99), weight_out=torch.full_like(cache["weight"], 5.5))
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=scale, **kw)
    full = any(n == cap and tl == TILE - 1 for n, tl in rows)
    assert int(cache.status) == (tra.DEV_CACHE_FULL if full else 0)
    o, bound = ref.step(q, kn, vn, scale)
    if apart:
        assert all(torch.equal(cache[n], own[n]) for n in own)
        got = kw["weight_out"].cpu().numpy()
        assert np.array_equal(kw["state_out"].cpu().numpy(), ref.t["state"])
        for b, (n, tl) in enumerate(rows):      # what lies behind a row's tokens is left alone
            m = 0 if n < 0 else n * TILE + tl + (0 if n == cap and tl == TILE - 1 else 1)
            assert np.all(got[b, :, m:] == 5.5)
            if n == cap and tl == TILE - 1:
                assert np.array_equal(got[b, :, :m], own["weight"][b, :, :m].cpu().numpy())
        ref.check_step(out, o, bound, kw["weight_out"], before)
        ref.same("k8", "v8", "sk", "sv", "table", "pos", "k_tail", "v_tail")
        # dropped and repeated, the step gives the same
        again, w2 = torch.empty_like(out), torch.empty_like(cache["weight"])
        tra.paged_attention_decode(cache, q, kn, vn, again, softmax_scale=scale, state_out=torch.empty_like(cache["state"]),
                                   weight_out=w2)
        act = [b for b in range(len(rows)) if (b, 0) in o]
        assert torch.equal(again[act], out[act])
        for b in act:
            m = rows[b][0] * TILE + rows[b][1] + 1
            assert torch.equal(w2[b, :, :m], kw["weight_out"][b, :, :m])
    else:
        ref.check_step(out, o, bound, None, before)
        ref.same()


@pytest.mark.parametrize("q_scale,v_scale", [(30.0, 1.0), (1e-3, 1e-9), (0.0, 1.0), (200.0, 1e6)])
def test_decode_ranges(q_scale, v_scale):
    """Peaked and flat rows, zero queries, scales of V that f16 cannot hold."""
    cache, (q, kn, vn) = _filled([(9, 20), (3, 63)], 8, 2, 128, 10, seed=1, v_scale=v_scale, q_scale=q_scale)
    if q_scale == 1e-3:
        q[0, 0] = (q[0, 0].float() * 1e-30).to(torch.bfloat16)
    ref = Mirror(cache)
    out = torch.empty_like(q)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.09)
    o, bound = ref.step(q, kn, vn, 0.09)
    ref.check_step(out, o, bound)
    ref.same()


@pytest.mark.parametrize("cap", [5, 20])
def test_decode_of_many_rows(cap):
    """More rows than CTAs, and than a warp scans at a time."""
    rows = [((3 * i) % 4, (7 * i) % 64) for i in range(75)]
    rows[40] = (-1, 0)
    cache, (q, kn, vn) = _filled(rows, 8, 4, 64, cap, seed=3)
    ref = Mirror(cache)
    out = torch.empty_like(q)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.125)
    o, bound = ref.step(q, kn, vn, 0.125)
    ref.check_step(out, o, bound)
    ref.same()


def test_decode_all_rows_idle():
    cache, (q, kn, vn) = _filled([(-1, 0), (-1, 5)], 4, 2, 64, 3, seed=3)
    ref = Mirror(cache)
    out = torch.full_like(q, 2.5)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.125)
    assert int(cache.status) == 0 and bool((out == 2.5).all())
    ref.same()


# ================================================================ evict
EVICTS = [
    # heads, d, cap, rows, keep, recent
    (8, 2, 128, 12, [(8, 17), (3, 5), (12, 0), (-1, 3), (4, 63)], 4, 0),
    (4, 4, 64, 40, [(30, 33), (20, 0), (33, 63), (11, 1)], 7, 90), (2, 1, 128, 9, [(8, 0)], 1, 0),
    (4, 2, 64, 70, [(64, 9)], 6, 10 ** 9), (8, 8, 128, 20, [(11, 20), (9, 2)], 8, 500), (4, 2, 128, 10, [(5, 60)], 5, 0),
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("hq,hkv,d,cap,rows,keep,recent", EVICTS, ids=str)
def test_evict(hq, hkv, d, cap, rows, keep, recent, ties):
    full = any(n > keep and n + keep > cap for n, _ in rows)
    cache, _ = _filled(rows, hq, hkv, d, cap, seed=cap, ties=ties)
    own = {n: x.clone() for n, x in cache.t.items()}
    ref = Mirror(cache)
    # into other arrays first: the cache's own stay, but for the new pages
    outs = {n + "_out": torch.full_like(cache[n], -5) for n in ("state", "table", "weight", "pos")}
    tra.paged_cache_evict(cache, keep=keep, recent=recent, **outs)
    assert int(cache.status) == (tra.DEV_CACHE_FULL if full else 0)
    ref.evict(keep, recent)
    assert all(torch.equal(cache[n], own[n]) for n in ("state", "table", "weight", "pos", "k_tail", "v_tail"))
    ref.same("k8", "v8", "sk", "sv")
    for n in ("state", "table"):
        assert np.array_equal(outs[n + "_out"].cpu().numpy(), ref.t[n]), n
    for n in ("weight", "pos"):
        got = outs[n + "_out"].cpu().numpy()
        for b in range(len(rows)):
            m = 0 if ref.t["state"][b, 0] < 0 else ref.t["state"][b, 0] * TILE + ref.t["state"][b, 1]
            assert np.array_equal(got[b, :, :m], ref.t[n][b, :, :m]), n
            assert np.all(got[b, :, m:] == -5), n
    # then in place, from the same start
    for n, x in own.items():
        cache[n].copy_(x)
    tra.paged_cache_evict(cache, keep=keep, recent=recent)
    ref.same()


def test_evict_of_many_tokens():
    """A row longer than the selection holds at a time, in place, and halves among its quotients."""
    cache, _ = _filled([(1000, 33)], 2, 1, 64, 1500, seed=8, ties=True)
    cache["sk"].fill_(0.0078125)      # equal scales: quotients of small whole numbers
    ref = Mirror(cache)
    tra.paged_cache_evict(cache, keep=400, recent=100)
    ref.evict(400, 100)
    ref.same()


def test_evict_pages_of_zero_and_tiny_scales():
    cache, _ = _filled([(6, 0)], 2, 2, 64, 10, seed=8)
    cache["sk"][::2] = 0.0
    cache["sv"][::3] = 1e-38          # values that are denormal in fp32
    ref = Mirror(cache)
    tra.paged_cache_evict(cache, keep=3)
    ref.evict(3, 0)
    ref.same()


def test_pages_past_32_bits():
    """A pool of more than 2^31 bytes, its last pages in use: the same as in a small pool."""
    rows, far = [(3, 63), (5, 10)], 270000
    near, (q, kn, vn) = _filled(rows, 8, 2, 128, 8, seed=5)
    n = near.n_pool
    t = dict(near.t)
    for name in ("k8", "v8", "sk", "sv"):
        x = near[name]
        t[name] = torch.zeros((far, *x.shape[1:]), dtype=x.dtype, device=DEV)
        t[name][far - n:].copy_(x)
    for name in ("state", "weight", "pos", "k_tail", "v_tail"):
        t[name] = near[name].clone()
    t["table"] = near["table"] + (far - n)
    big = tra.PagedCache(2, 8, 2, 128, 8, tensors=t)
    assert t["k8"].numel() > 2 ** 31
    gen = _rng(2)
    k, v = _normal(gen, 400, 2, 128), _normal(gen, 400, 2, 128)
    shape = tra.Shape([0, 270, 400], 8, 2, 128)
    for call in ("decode", "evict", "fill"):
        outs = []
        for c in (near, big):
            if call == "decode":
                outs.append(torch.empty_like(q))
                tra.paged_attention_decode(c, q, kn, vn, outs[-1], softmax_scale=0.09)
            elif call == "evict":
                tra.paged_cache_evict(c, keep=2, recent=40)
            else:
                tra.paged_cache_fill(c, shape, k, v, keep=3)
        if outs:
            assert torch.equal(*outs)
        assert int(near.status) == 0 and int(big.status) == 0
        assert torch.equal(near["table"] + (far - n), big["table"])
        for name in near.NAMES:
            if name != "table":
                assert torch.equal(near[name], big[name][-n:] if name in ("k8", "v8", "sk", "sv") else big[name]), (call, name)


def test_decode_of_millions_of_pages():
    """64 rows of 70,000 pages (a list of more than 2^22 items), all of them the same four: attention over four
    pages with multiplicities.  (Reading shared pages is all this step does: no tail is full.)"""
    B, n, d, scale = 64, 70000, 64, 0.125
    gen = _rng(11)
    z = lambda *s, t=torch.float32: torch.zeros(s, device=DEV, dtype=t)  # noqa: E731
    t = dict(k8=torch.randint(-127, 128, (4, TILE, d), generator=gen, device=DEV, dtype=torch.int8),
             v8=torch.randint(-127, 128, (4, TILE, d), generator=gen, device=DEV, dtype=torch.int8),
             sk=torch.rand(4, generator=gen, device=DEV) * 0.02 + 0.005, sv=torch.rand(4, generator=gen, device=DEV) * 0.05,
             table=(torch.arange(n, device=DEV, dtype=torch.int32) % 4).repeat(B, 1, 1).contiguous(), state=z(B, 4, t=torch.int32),
             weight=z(B, 1, (n + 1) * TILE), pos=z(B, 1, (n + 1) * TILE, t=torch.int32),
             k_tail=z(B, 1, TILE, d, t=torch.bfloat16), v_tail=z(B, 1, TILE, d, t=torch.bfloat16))
    t["state"][:, 0] = n
    cache = tra.PagedCache(B, 1, 1, d, n, tensors=t)
    q, kn, vn = _normal(gen, B, 1, d), _normal(gen, B, 1, d), _normal(gen, B, 1, d)
    out = torch.empty_like(q)
    tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=scale)
    assert int(cache.status) == 0
    k = (t["k8"].double() * t["sk"].double()[:, None, None]).view(-1, d)
    v = (t["v8"].double() * t["sv"].double()[:, None, None]).view(-1, d)
    s = torch.cat([q[:, 0].double() @ k.T, (q[:, 0].double() * kn[:, 0].double()).sum(1, keepdim=True)], 1) * scale
    many = torch.cat([torch.full((256,), n / 4, device=DEV, dtype=torch.float64), torch.ones(1, device=DEV, dtype=torch.float64)])
    p = torch.exp(s - s.amax(1, keepdim=True))
    p = p / (p * many).sum(1, keepdim=True)
    o = (p[:, :256] * (n / 4)) @ v + p[:, 256:] * vn[:, 0].double()
    # the sums: a warp adds 8 terms of each of its pages, a quarter of a piece's, one after another in fp32
    rel = 8 * (n * B / 296) / 4 * 2.0 ** -24 + 2.0 ** -17
    mag = (p[:, :256] * (n / 4)) @ v.abs() + p[:, 256:] * vn[:, 0].double().abs()
    assert bool(((out[:, 0].double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -10.9 + 2 * rel) * mag).all())
    w = cache["weight"][:, 0, :n * TILE + 1].double()
    assert bool(((w[:, :-1].view(B, n // 4, 256) - p[:, None, :256]).abs() <= 2 * rel * p[:, None, :256]).all())
    assert bool(((w[:, -1] - p[:, 256]).abs() <= 2 * rel * p[:, 256]).all())
    assert bool((cache["state"][:, :3] == torch.tensor([n, 1, 1], device=DEV)).all())


# ================================================================ states and pages out of range
@pytest.mark.parametrize("state", [(4, 0), (2, 64), (2, -1)])
def test_bad_states_are_reported_and_left(state):
    for call in ("decode", "evict"):
        cache, (q, kn, vn) = _filled([(2, 7), (2, 7)], 4, 2, 64, 3, seed=1)
        cache["state"][0, 0], cache["state"][0, 1] = state
        ref = Mirror(cache)
        out = torch.zeros_like(q)
        if call == "decode":
            tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1)
        else:
            tra.paged_cache_evict(cache, keep=1)
        assert int(cache.status) == tra.DEV_BAD_CACHE
        assert not bool(out[0].any())
        assert np.array_equal(cache["state"][0].cpu().numpy(), ref.t["state"][0])
        for n in ("weight", "pos", "table", "k_tail", "v_tail"):
            x = cache[n][0].float().cpu().numpy()
            assert np.array_equal(x, ref.t[n][0]), n


@pytest.mark.parametrize("bad", [-1, 1 << 20, 2 ** 31 - 1, -2 ** 31])
def test_bad_pages_are_reported(bad):
    """No page outside the pool is read or written; the other rows go on."""
    for call in ("fill", "decode", "evict", "decode new"):
        cache, (q, kn, vn) = _filled([(2, 63), (2, 7)], 4, 2, 64, 4, seed=1)
        cache["table"][0, 1, {"fill": 0, "decode": 1, "evict": 0, "decode new": 2}[call]] = bad
        ref = Mirror(cache)
        out = torch.zeros_like(q)
        if call == "fill":
            gen = _rng(1)
            k, v = _normal(gen, 300, 2, 64), _normal(gen, 300, 2, 64)
            tra.paged_cache_fill(cache, tra.Shape([0, 150, 300], 4, 2, 64), k, v, keep=2)
        elif call == "evict":
            tra.paged_cache_evict(cache, keep=1)
        else:
            tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1)
        assert int(cache.status) == tra.DEV_BAD_CACHE, call
        if call.startswith("decode"):
            ref.t["table"][0, 1] = ref.t["table"][1, 1]
            o, bound = ref.step(q, kn, vn, 0.1)
            good = {key: x for key, x in o.items() if key == (1, 0) or key == (1, 1) or key == (0, 0)}
            ref.check_step(out, good, bound)


# ================================================================ together
def test_cache_from_prompt_to_eviction():
    """Weights of a prompt, the cache filled by them, decoded past page borders and cut in between: the
    definitions' results after every call."""
    hq, hkv, d, lens = 8, 2, 128, [500, 200, 64]
    gen, cu = _rng(17), _cu(lens)
    q, k, v = (_normal(gen, cu[-1], h, d) for h in (hq, hkv, hkv))
    shape, scale = tra.Shape(cu, hq, hkv, d), 1.0 / math.sqrt(d)
    plan = api.EvictingDecodePlan(shape, keep=3, limit=5, recent=70, n_queries=64)
    w = plan.prefill(q, k, v)
    ref = Mirror(plan.cache)
    ref.fill(cu, k, v, w, 3, 70)
    ref.same("state", "table", "pos", "weight", "sk", "sv")
    ref.pull()
    seen_evictions = 0
    for i in range(200):
        qs, kn, vn = (_normal(gen, 3, h, d) for h in (hq, hkv, hkv))
        if any(n >= 5 and t == 63 for n, t in plan.rows):
            ref.evict(3, 70)
            seen_evictions += 1
        out = torch.empty_like(qs)
        plan.step(qs, kn, vn, out)
        o, bound = ref.step(qs, kn, vn, scale)
        ref.check_step(out, o, bound)
        if i % 40 == 39 or any(t == 0 for _, t in plan.rows):
            ref.same()
        assert plan.cache["state"][:, :2].cpu().tolist() == plan.rows
    # the first row has 3 pages and 52 tokens: 5 pages and 63 tokens after 139 steps, and again 128 later
    assert seen_evictions == 1 and int(plan.status) == 0


def test_captured_steps():
    """A captured step and eviction, replayed, do what the calls do."""
    rows = [(3, 62), (5, 10)]
    a, (q, kn, vn) = _filled(rows, 8, 2, 128, 9, seed=5)
    b, _ = _filled(rows, 8, 2, 128, 9, seed=5)
    outs = [torch.empty_like(q) for _ in range(2)]

    def work(cache, out):
        tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.09)
        tra.paged_cache_evict(cache, keep=4, recent=10)

    warm, _ = _filled(rows, 8, 2, 128, 9, seed=5)
    work(warm, torch.empty_like(q))
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work(a, outs[0])
    for i in range(3):
        q.copy_(_normal(_rng(i), *q.shape))
        g.replay()
        torch.cuda.synchronize()
        work(b, outs[1])
        assert torch.equal(outs[0], outs[1])
        for n in a.NAMES:
            assert torch.equal(a[n], b[n]), n


def test_captured_prompt():
    """Weight sums and a fill from them, captured and replayed on other inputs."""
    lens = [300, 64, 777]
    cu, gen = _cu(lens), _rng(4)
    shape, n = tra.Shape(cu, 8, 2, 128), sum(lens)
    q, k, v = (_normal(gen, n, h, 128) for h in (8, 2, 2))
    made = []
    for _ in range(2):
        cache, _ = _filled([(-1, 0)] * 3, 8, 2, 128, 6, seed=1)
        made.append((cache, torch.zeros(n, 2, device=DEV), torch.zeros(8, n, device=DEV)))

    def work(cache, w, lse):
        tra.attention_weight_sums(shape, q, k, w, lse, n_queries=64, softmax_scale=0.09)
        tra.paged_cache_fill(cache, shape, k, v, keep=4, recent=20, weights=w)

    work(*made[1])
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work(*made[0])
    for i in range(3):
        q.copy_(_normal(_rng(i), *q.shape))
        v.copy_(_normal(_rng(10 + i), *v.shape))
        g.replay()
        torch.cuda.synchronize()
        work(*made[1])
        for a, b in zip(made[0][1:], made[1][1:]):
            assert torch.equal(a, b)
        for name in made[0][0].NAMES:
            assert torch.equal(made[0][0][name], made[1][0][name]), name


def test_streams():
    """Two caches stepped on two streams at once, and weight sums on a stream of its own."""
    made = [_filled([(60, 20), (33, 63)], 8, 8, 128, 64, seed=s) for s in (1, 2)]
    refs, streams = [Mirror(c) for c, _ in made], [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(st[0]) for _, st in made]
    gen = _rng(6)
    q, k = _normal(gen, 900, 4, 64), _normal(gen, 900, 2, 64)
    shape = tra.Shape([0, 900], 4, 2, 64)
    w, lse = torch.empty(900, 2, device=DEV), torch.empty(4, 900, device=DEV)
    int(shape.status)
    torch.cuda.synchronize()
    for (c, st), out, s in zip(made, outs, streams):
        tra.paged_attention_decode(c, *st, out, softmax_scale=0.09, stream=s)
    tra.attention_weight_sums(shape, q, k, w, lse, softmax_scale=0.125, stream=streams[2])
    with torch.cuda.stream(streams[2]):
        w2, l2 = torch.empty_like(w), torch.empty_like(lse)
        tra.attention_weight_sums(shape, q, k, w2, l2, softmax_scale=0.125)
    torch.cuda.synchronize()
    for (c, st), out, ref in zip(made, outs, refs):
        o, bound = ref.step(*st, 0.09)
        ref.check_step(out, o, bound)
        ref.same()
    ref, _, size = _sums64(q, k, [0, 900], 0, 0.125)
    assert torch.equal(w, w2)
    assert bool((w.double() - ref).abs().le(_weight_bounds(size, lse)[0] * ref + 1e-30).all())


def test_python_refusals():
    cache, (q, kn, vn) = _filled([(2, 7)], 4, 2, 64, 4, seed=1)
    out = torch.empty_like(q)
    ok = dict(q=q, kn=kn, vn=vn, out=out)
    for name, bad in (("q", q.float()), ("q", q[:, :2]), ("kn", kn.transpose(1, 2)), ("vn", vn.cpu()), ("out", out[:, :1]),
                      ("q", q.expand(2, -1, -1))):
        a = ok | {name: bad}
        with pytest.raises(tra.TraError):
            tra.paged_attention_decode(cache, a["q"], a["kn"], a["vn"], a["out"], softmax_scale=0.1)
    with pytest.raises(tra.TraError):
        tra.paged_attention_decode(cache, q, kn, vn, out, softmax_scale=0.1, weight_out=cache["weight"][:, :, :64])
    with pytest.raises(tra.TraError):
        tra.paged_cache_evict(cache, keep=1, state_out=torch.empty_like(cache["state"]))
    with pytest.raises(tra.TraError):
        tra.paged_cache_evict(cache, keep=5)
    shape = tra.Shape([0, 128], 4, 2, 64)
    k = torch.zeros(128, 2, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(weights=torch.zeros(128, 2, device=DEV, dtype=torch.float64)), dict(keep=9), dict(recent=-1)):
        with pytest.raises(tra.TraError):
            tra.paged_cache_fill(cache, shape, k, k, **({"keep": 2} | kw))
    with pytest.raises(tra.TraError):
        tra.paged_cache_fill(cache, tra.Shape([0, 64, 128], 4, 2, 64), k, k, keep=2)   # two sequences, one row
