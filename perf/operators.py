"""The cases on which the evicting key/value cache and its weight sums are timed, with their plain forms.

Four operators, named by a case's "op":

weights  accumulated attention weight of a prompt's keys: with lse[h, i] the logarithm of the sum over
         j <= i of exp(scale q_i . k_j), w[j, g] = the sum over the query heads h of KV head g and the
         window's queries i >= j of exp(scale q_i . k_j - lse[h, i])
fill     a prompt's K and V into a paged 8-bit cache that keeps the tokens of highest weight
step     one decode step over that cache: attention, the weights it gives to the cached tokens, and the
         append of the new token (a tail of 64 tokens becomes a page)
evict    a cache shrunk to its tokens of highest weight

A page is 64 tokens of one sequence and one KV head: int8 codes with one scale for K and one for V,
s = fl32(max |x| / 127), code = round-half-even(fl32(x / s)).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
#: largest score matrix the plain form holds at a time (elements)
CHUNK = 1 << 28
HEADS = ("32/8", "28/4", "8/8", "16/2", "12/4", "4/4", "2/2", "8/1")


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the weights of a short prompt, every query counted: where the launches count
        dict(name="weights_t256", op="weights", heads="2/2", d=64, B=1, T=256, ragged=False, window=0, given=False),
        # an 8K prompt whose last 64 queries decide what is kept: the usual cheap form before decoding
        dict(name="weights_t8k_last64", op="weights", heads="32/8", d=128, B=1, T=8192, ragged=False, window=64, given=False),
        # a ragged batch of prompts, every query counted and the normalisers computed as well
        dict(name="weights_varlen8_all", op="weights", heads="28/4", d=128, B=8, T=6133, ragged=True, window=0, given=False),
        # a 32K prompt, every query, with the normalisers that its prefill left
        dict(name="weights_t32k_all", op="weights", heads="32/8", d=128, B=1, T=32768, ragged=False, window=0, given=True),
        # an 8K prompt cut to 2K tokens per head
        dict(name="fill_t8k_keep2k", op="fill", heads="32/8", d=128, B=1, T=8192, ragged=False, keep=32, recent=128),
        # a ragged batch of 16 prompts of up to 32K tokens, each cut to at most 8K per head
        dict(name="fill_b16_32k_keep8k", op="fill", heads="32/8", d=128, B=16, T=32749, ragged=True, keep=128, recent=256),
        # one sequence over a 2K cache: the step's latency
        dict(name="step_b1_2k", op="step", heads="32/8", d=128, B=1, T=2048 + 17, ragged=False),
        # a ragged serving batch, full tails that become pages and an idle row among it
        dict(name="step_b24_ragged", op="step", heads="28/4", d=128, B=24, T=8192 + 63, ragged=True),
        # the decode benchmark's batch and context, all of it kept
        dict(name="step_b16_32k", op="step", heads="32/8", d=128, B=16, T=32768 + 40, ragged=False),
        # one sequence of small heads, 4K tokens to 2K
        dict(name="evict_b1_4k_d64", op="evict", heads="8/8", d=64, B=1, T=4096 + 5, ragged=False, keep=32, recent=64),
        # the serving batch, ragged, to 4K tokens per head (rows that are shorter stay as they are)
        dict(name="evict_b24_ragged", op="evict", heads="28/4", d=128, B=24, T=8192 + 63, ragged=True, keep=64, recent=128),
        # 16 sequences of 32K tokens to 16K
        dict(name="evict_b16_32k", op="evict", heads="32/8", d=128, B=16, T=32768 + 40, ragged=False, keep=256, recent=256),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("weights", "fill", "step", "evict"))
    case = dict(op=op, heads=rng.choice(HEADS), d=rng.choice((64, 128)), ragged=rng.random() < 0.5)
    if op == "weights":
        T = _spread(rng, 1, 16384)
        case |= dict(B=_spread(rng, 1, max(1, min(8, 16384 // T))), T=T, window=rng.choice((0, 0, 1, _spread(rng, 2, 512))),
                     given=rng.random() < 0.5)
    elif op == "fill":
        T = _spread(rng, 1, 32768)
        case |= dict(B=_spread(rng, 1, max(1, min(16, 262144 // T))), T=T, keep=_spread(rng, 1, 128), recent=rng.choice((0, 32, 300)))
    else:
        T = _spread(rng, 64 if op == "evict" else 1, 32768)
        case |= dict(B=_spread(rng, 1, max(1, min(32, 262144 // T))), T=T)
        if op == "evict":
            case |= dict(keep=max(1, int((T // BLOCK) * rng.uniform(0.1, 0.9))), recent=rng.choice((0, 64, 500)))
    return case


def _heads(case):
    hq, hkv = case["heads"].split("/")
    return int(hq), int(hkv)


def _lengths(case):
    """Tokens of each sequence: equal, or falling from T to about 3/8 T."""
    B, T = case["B"], case["T"]
    return [max(1, T - (5 * b * T) // (8 * B)) for b in range(B)] if case["ragged"] else [T] * B


def _rows(case):
    """(pages, tail) of each sequence of a cache: T tokens, a ragged batch shorter row by row, with an idle row in the
    middle of a batch of eight or more."""
    rows = [(t // BLOCK, t % BLOCK) for t in _lengths(case)]
    if case["ragged"] and case["B"] >= 8:
        rows[case["B"] // 2] = (-1, 0)
    return rows


def _cap(case):
    """Page table entries of a row: the longest row, and room for one step's page or an eviction's survivors."""
    return max(1, case["T"] // BLOCK) + (case["keep"] if case["op"] == "evict" else 1)


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _normal(gen, ntok, H, d, outliers):
    """bf16 N(0, 1), with four channels per head of ten times the size where outliers are asked for."""
    x = _randn(gen, ntok, H, d)
    if outliers:
        ch = torch.rand((H, d), generator=gen, device="cuda").argsort(1)[:, :4]
        f = torch.ones((H, d), device="cuda").scatter_(1, ch, 10.0)
        x *= f
    return x.to(torch.bfloat16)


def _heavy(gen, *shape):
    """Weights as they accumulate: heavy-tailed, with a share of tokens that nothing has looked at (ties at zero)."""
    x = torch.exp(2.5 * _randn(gen, *shape) - 3.0)
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.05, torch.zeros_like(x), x)


def _quantised(x):
    """x fp32 [..., 64, d] as int8 codes and one fp32 scale per block."""
    top = x.abs().amax((-2, -1))
    s = top / torch.full_like(top, 127.0)  # a tensor: by a number torch multiplies with its reciprocal, which rounds twice
    safe = torch.where(s > 0, s, torch.ones_like(s))
    return torch.round(x / safe[..., None, None]).clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    gen = _gen(seed)
    hq, hkv = _heads(case)
    d, B = case["d"], case["B"]
    st = dict(case=case, hq=hq, hkv=hkv, scale=1.0 / math.sqrt(d))
    if case["op"] in ("weights", "fill"):
        lens = _lengths(case)
        cu = [0]
        for t in lens:
            cu.append(cu[-1] + t)
        st |= dict(cu=cu, k=_normal(gen, cu[-1], hkv, d, True))
        if own:
            import tile_routed_mixed_causal_b200 as tra
            st["shape"] = tra.Shape(cu, hq, hkv, d)
    if case["op"] == "weights":
        st["q"] = _normal(gen, cu[-1], hq, d, True)
        st["weights"] = torch.zeros((cu[-1], hkv), device="cuda")
        st["lse"] = torch.zeros((hq, cu[-1]), device="cuda")
        if case["given"]:
            st["lse"].copy_(_weights_plain(st, False)[1])
        return st
    if case["op"] == "fill":
        cap = case["keep"]
        st["v"] = _normal(gen, cu[-1], hkv, d, False)
        st["importance"] = _heavy(gen, cu[-1], hkv)
    else:
        cap = _cap(case)
    n_pool = B * hkv * cap
    z = lambda *s, t=torch.float32: torch.zeros(s, device="cuda", dtype=t)  # noqa: E731
    st |= dict(k8=z(n_pool, BLOCK, d, t=torch.int8), v8=z(n_pool, BLOCK, d, t=torch.int8), sk=z(n_pool), sv=z(n_pool),
               table=torch.randperm(n_pool, generator=gen, device="cuda").to(torch.int32).view(B, hkv, cap),
               state=z(B, 4, t=torch.int32), weight=z(B, hkv, (cap + 1) * BLOCK), pos=z(B, hkv, (cap + 1) * BLOCK, t=torch.int32),
               k_tail=z(B, hkv, BLOCK, d, t=torch.bfloat16), v_tail=z(B, hkv, BLOCK, d, t=torch.bfloat16))
    if case["op"] != "fill":
        for b, (n, tail) in enumerate(_rows(case)):
            st["state"][b] = torch.tensor([n, tail, max(0, n) * 2 * BLOCK + tail, 0], dtype=torch.int32)
            m = max(0, n) * BLOCK + tail
            st["weight"][b, :, :m] = _heavy(gen, hkv, m)
            # positions of tokens that an earlier eviction left: ascending, with gaps
            st["pos"][b, :, :m] = torch.cumsum(torch.randint(1, 3, (hkv, m), generator=gen, device="cuda"), 1).to(torch.int32)
            st["k_tail"][b] = _normal(gen, BLOCK, hkv, d, True).transpose(0, 1)
            st["v_tail"][b] = _normal(gen, BLOCK, hkv, d, False).transpose(0, 1)
            if n > 0:
                ids = st["table"][b, :, :n].long()
                for codes, scales, out in (("k8", "sk", True), ("v8", "sv", False)):
                    x = _normal(gen, n * BLOCK, hkv, d, out).float().transpose(0, 1).reshape(hkv, n, BLOCK, d)
                    st[codes][ids], st[scales][ids] = _quantised(x)
    if case["op"] == "step":
        st |= dict(q=_normal(gen, B, hq, d, True), k_new=_normal(gen, B, hkv, d, True), v_new=_normal(gen, B, hkv, d, False),
                   out=z(B, hq, d, t=torch.bfloat16), state_out=z(B, 4, t=torch.int32), weight_out=z(B, hkv, (cap + 1) * BLOCK))
    if case["op"] == "evict":
        st |= {n + "_out": torch.zeros_like(st[n]) for n in ("table", "state", "weight", "pos")}
    if own:
        import tile_routed_mixed_causal_b200 as tra
        st["cache"] = tra.PagedCache(B, hq, hkv, d, cap, tensors={n: st[n] for n in (
            "k8", "v8", "sk", "sv", "table", "state", "weight", "pos", "k_tail", "v_tail")})
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _weights_plain(st, with_sums=True):
    """(weights, lse) of the window's queries; lse rows outside the window stay zero."""
    case, cu, hkv = st["case"], st["cu"], st["hkv"]
    grp, given = st["hq"] // hkv, case["given"] and with_sums
    w, lse = torch.zeros_like(st["weights"]), torch.zeros_like(st["lse"])
    for t0, t1 in zip(cu, cu[1:]):
        T = t1 - t0
        i0 = max(0, T - case["window"]) if case["window"] else 0
        rows = max(1, CHUNK // (grp * T))
        for g in range(hkv):
            hs = slice(g * grp, (g + 1) * grp)
            kk = st["k"][t0:t1, g].float()
            for a in range(i0, T, rows):
                e = min(T, a + rows)
                s = torch.matmul(st["q"][t0 + a:t0 + e, hs].float().transpose(0, 1), kk[:e].t()) * st["scale"]
                s.masked_fill_(torch.arange(e, device="cuda")[None, :] > torch.arange(a, e, device="cuda")[:, None], -math.inf)
                if given:
                    lz = st["lse"][hs, t0 + a:t0 + e]
                else:
                    m = s.amax(-1)
                    lz = m + torch.log(torch.exp(s - m[..., None]).sum(-1))
                lse[hs, t0 + a:t0 + e] = lz
                if with_sums:
                    w[t0:t0 + e, g] += torch.exp(s.sub_(lz[..., None])).sum((0, 1))
    return w, lse


def _kept(weight, protected, count):
    """The count indices of highest weight along the last axis (protected ones first, ties to the lower), ascending."""
    x = torch.where(protected, math.inf, weight)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :count]
    return torch.sort(order, dim=-1).values


def _fill_plain(st):
    case, hkv = st["case"], st["hkv"]
    d = case["d"]
    for b, (t0, t1) in enumerate(zip(st["cu"], st["cu"][1:])):
        T = t1 - t0
        nb, tail = T // BLOCK, T % BLOCK
        n = min(nb, case["keep"])
        body, m = nb * BLOCK, n * BLOCK
        st["state"][b] = torch.tensor([n, tail, T, 0], dtype=torch.int32, device="cuda")
        imp = st["importance"][t0:t1].t()
        if n:
            first = max(T - case["recent"], body - m)
            idx = _kept(imp[:, :body], (torch.arange(body, device="cuda") >= first)[None, :], m)
            st["weight"][b, :, :m] = imp.gather(1, idx)
            st["pos"][b, :, :m] = idx.to(torch.int32)
            ids = st["table"][b, :, :n].long()
            for x, codes, scales in (("k", "k8", "sk"), ("v", "v8", "sv")):
                rows = st[x][t0:t1].transpose(0, 1).gather(1, idx[..., None].expand(-1, -1, d)).float()
                st[codes][ids], st[scales][ids] = _quantised(rows.view(hkv, n, BLOCK, d))
        st["weight"][b, :, m:m + tail] = imp[:, body:]
        st["pos"][b, :, m:m + tail] = torch.arange(body, T, device="cuda", dtype=torch.int32)
        st["k_tail"][b, :, :tail] = st["k"][t0 + body:t1].transpose(0, 1)
        st["v_tail"][b, :, :tail] = st["v"][t0 + body:t1].transpose(0, 1)


def _step_plain(st):
    case, hkv = st["case"], st["hkv"]
    B, d, grp = case["B"], case["d"], st["hq"] // hkv
    state = st["state"]
    n, tl, active = state[:, 0].long(), state[:, 1].long(), state[:, 0] >= 0
    st["state_out"].copy_(state)
    most = (st["table"].shape[-1] - 1)
    ids = st["table"][:, :, :most].long()
    b_of = torch.nonzero(active).flatten()
    st["k_tail"][b_of, :, tl[b_of]] = st["k_new"][b_of]
    st["v_tail"][b_of, :, tl[b_of]] = st["v_new"][b_of]
    st["pos"][b_of, :, (n * BLOCK + tl)[b_of]] = state[b_of, 2:3]
    # scores over [pages | tail], the slots past each row's pages and tail masked
    q = st["q"].float().view(B, hkv, grp, d)
    x = (st["k8"][ids].float() * st["sk"][ids][..., None, None]).reshape(B, hkv, most * BLOCK, d)
    s = torch.cat([torch.matmul(q, x.transpose(-1, -2)), torch.matmul(q, st["k_tail"].float().transpose(-1, -2))], -1) * st["scale"]
    slot = torch.arange(most * BLOCK + BLOCK, device="cuda")
    live = torch.where(slot < most * BLOCK, slot[None, :] < n[:, None] * BLOCK, slot[None, :] - most * BLOCK <= tl[:, None])
    s.masked_fill_(~live[:, None, None, :], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    x = (st["v8"][ids].float() * st["sv"][ids][..., None, None]).reshape(B, hkv, most * BLOCK, d)
    o = torch.matmul(p[..., :most * BLOCK], x) + torch.matmul(p[..., most * BLOCK:], st["v_tail"].float())
    st["out"][b_of] = o.reshape(B, hkv * grp, d)[b_of].to(torch.bfloat16)
    # weights in the cache's order: pages, then the tail behind the last one; the new token starts from nothing
    at = torch.where(slot < most * BLOCK, slot[None, :], slot[None, :] - most * BLOCK + n[:, None] * BLOCK)
    bi, si = torch.nonzero(live & active[:, None], as_tuple=True)
    old = torch.where((si == most * BLOCK + tl[bi])[:, None], 0.0, st["weight"][bi, :, at[bi, si]])
    st["weight_out"][bi, :, at[bi, si]] = old + p.sum(2)[bi, :, si]
    full = torch.nonzero(active & (tl == BLOCK - 1)).flatten()
    for name, codes, scales in (("k_tail", "k8", "sk"), ("v_tail", "v8", "sv")):
        page = st["table"][full, :, n[full]].long()
        st[codes][page], st[scales][page] = _quantised(st[name][full].float())
    new = torch.stack([n + (tl == BLOCK - 1), (tl + 1) % BLOCK, state[:, 2] + 1, state[:, 3]], 1).to(torch.int32)
    st["state_out"].copy_(torch.where(active[:, None], new, state))


def _evict_plain(st):
    case, hkv = st["case"], st["hkv"]
    d, keep = case["d"], case["keep"]
    for name in ("table", "state", "weight", "pos"):
        st[name + "_out"].copy_(st[name])
    for b, (n, tail) in enumerate(_rows(case)):
        if n <= keep:
            continue
        body, m = n * BLOCK, keep * BLOCK
        first = max(body + tail - case["recent"], body - m)
        idx = _kept(st["weight"][b, :, :body], (torch.arange(body, device="cuda") >= first)[None, :], m)
        row = st["table"][b]
        src, dst = row[:, :n].long(), row[:, n:n + keep].long()
        for codes, scales in (("k8", "sk"), ("v8", "sv")):
            x = (st[codes][src].float() * st[scales][src][..., None, None]).view(hkv, body, d)
            x = x.gather(1, idx[..., None].expand(-1, -1, d)).view(hkv, keep, BLOCK, d)
            st[codes][dst], st[scales][dst] = _quantised(x)
        st["table_out"][b] = torch.cat([row[:, n:n + keep], row[:, :n], row[:, n + keep:]], 1)
        for name in ("weight", "pos"):
            st[name + "_out"][b, :, :m + tail] = torch.cat([st[name][b, :, :body].gather(1, idx), st[name][b, :, body:body + tail]], 1)
            st[name + "_out"][b, :, m + tail:] = 0
        st["state_out"][b, 0] = keep


def run(st):
    op = st["case"]["op"]
    case = st["case"]
    if own:
        import tile_routed_mixed_causal_b200 as tra
        if op == "weights":
            tra.attention_weight_sums(st["shape"], st["q"], st["k"], st["weights"], st["lse"], n_queries=case["window"],
                                      softmax_scale=st["scale"], lse_given=case["given"])
            return {"weights": st["weights"], "lse": st["lse"]}
        cache = st["cache"]
        if op == "fill":
            tra.paged_cache_fill(cache, st["shape"], st["k"], st["v"], keep=case["keep"], recent=case["recent"],
                                 weights=st["importance"])
        elif op == "step":
            tra.paged_attention_decode(cache, st["q"], st["k_new"], st["v_new"], st["out"], softmax_scale=st["scale"],
                                       state_out=st["state_out"], weight_out=st["weight_out"])
        else:
            tra.paged_cache_evict(cache, keep=case["keep"], recent=case["recent"], state_out=st["state_out"],
                                  table_out=st["table_out"], weight_out=st["weight_out"], pos_out=st["pos_out"])
    elif op == "weights":
        w, lse = _weights_plain(st)
        return {"weights": w, "lse": lse}
    elif op == "fill":
        _fill_plain(st)
    elif op == "step":
        _step_plain(st)
    else:
        _evict_plain(st)
    # the codes are whole numbers of their page's scale and have to be equal
    pages = {n: st[n] for n in ("k8", "v8", "sk", "sv")}
    if op == "fill":
        return pages | {n: st[n] for n in ("state", "weight", "pos", "k_tail", "v_tail")}
    if op == "step":
        return pages | {n: st[n] for n in ("out", "state_out", "weight_out", "pos", "k_tail", "v_tail")}
    return pages | {n + "_out": st[n + "_out"] for n in ("table", "state", "weight", "pos")}


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    hq, hkv = _heads(case)
    d, keep = case["d"], case.get("keep", 0)
    if case["op"] == "weights":
        lens = _lengths(case)
        wins = [min(t, case["window"] or t) for t in lens]
        pairs = sum(w * t - w * (w - 1) // 2 for w, t in zip(wins, lens))
        # q of the window, k, the sums, the normalisers; one product of every query with its keys
        return {"bytes": sum(wins) * hq * (2 * d + 4) + sum(lens) * hkv * (2 * d + 4), "flops": 2 * d * pairs * hq}
    if case["op"] == "fill":
        lens = _lengths(case)
        kept = sum(min(t // BLOCK, keep) * BLOCK for t in lens)
        tails = sum(t % BLOCK for t in lens)
        # every weight; K and V of the kept in, codes, weights and positions out; tails copied
        return {"bytes": hkv * (4 * sum(lens) + kept * (4 * d + 2 * d + 8) + tails * (8 * d + 8)), "flops": 0}
    rows = [r for r in _rows(case) if r[0] >= 0]
    if case["op"] == "step":
        tok, tails = sum(n * BLOCK for n, _ in rows), sum(t + 1 for _, t in rows)
        pages = sum(n for n, _ in rows)
        # codes, scales and page numbers once, weights in and out, the tails, q and out
        return {"bytes": hkv * (tok * (2 * d + 8) + 12 * pages + tails * (4 * d + 8)) + len(rows) * (4 * hq * d),
                "flops": 4 * d * hq * (tok + tails)}
    cut = [r for r in rows if r[0] > keep]
    kept = len(cut) * keep * BLOCK
    # every weight of the rows that shrink; the survivors' codes in and out, their weights and positions
    return {"bytes": hkv * (4 * sum(n * BLOCK for n, _ in cut) + kept * (4 * d + 12)), "flops": 0}


# ------------------------------------------------------------------------------------------ in 64 bits
def _lexkept(weight, first, count):
    """As the definition orders them: from `first` on before all others, then by falling weight, then by index."""
    j = np.arange(weight.shape[0])
    order = np.lexsort((j, -weight.astype(np.float64), j < first))
    return np.sort(order[:count])


def _codes64(x):
    """Codes (int8) and scales (fp32) of the blocks x float64 [n, 64, d]: the scale and the quotient are rounded to fp32
    by the definition, everything else is exact."""
    s = (x.abs().flatten(1).max(1).values / 127.0).float()
    q = (x / torch.where(s == 0, 1.0, s.double())[:, None, None]).float()
    return torch.round(q).clamp(-127, 127).to(torch.int8), s


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv = st["hq"], st["hkv"]
    grp, d, scale = hq // hkv, case["d"], 1.0 / math.sqrt(case["d"])
    if case["op"] == "weights":
        w = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
        for t0, t1 in zip(st["cu"], st["cu"][1:]):
            T = t1 - t0
            lo = T - min(T, case["window"] or T)
            for h in range(hq):
                kk = st["k"][t0:t1, h // grp].double()
                step = max(1, (CHUNK // 4) // T)
                for a in range(lo, T, step):
                    e = min(a + step, T)
                    s = st["q"][t0 + a:t0 + e, h].double() @ kk[:e].T * scale
                    s = torch.tril(torch.exp(s), diagonal=a) if not case["given"] else s
                    if case["given"]:
                        z = st["lse"][h, t0 + a:t0 + e].double()
                        p = torch.tril(torch.exp(s - z[:, None]), diagonal=a)
                    else:
                        z = torch.log(s.sum(1))
                        p = s * torch.exp(-z)[:, None]
                    lse[h, t0 + a:t0 + e] = z
                    w[t0:t0 + e, h // grp] += p.sum(0)
        return {"weights": w, "lse": lse}
    if case["op"] == "fill":
        for b, (t0, t1) in enumerate(zip(st["cu"], st["cu"][1:])):
            T = t1 - t0
            n = min(T // BLOCK, case["keep"])
            body = T // BLOCK * BLOCK
            st["state"][b] = torch.tensor([n, T - body, T, 0])
            imp = st["importance"][t0:t1].cpu().numpy()
            for g in range(hkv):
                kept = _lexkept(imp[:body, g], max(T - case["recent"], body - n * BLOCK), n * BLOCK)
                at = np.concatenate([kept, np.arange(body, T)])
                idx = torch.from_numpy(at).cuda()
                st["pos"][b, g, :len(at)] = idx.int()
                st["weight"][b, g, :len(at)] = st["importance"][t0:t1, g][idx]
                for x, codes, scales, tail in (("k", "k8", "sk", "k_tail"), ("v", "v8", "sv", "v_tail")):
                    rows = st[x][t0:t1, g][idx]
                    st[tail][b, g, :T - body] = rows[n * BLOCK:]
                    if n:
                        page = st["table"][b, g, :n].long()
                        st[codes][page], st[scales][page] = _codes64(rows[:n * BLOCK].double().view(n, BLOCK, d))
        return {n: st[n] for n in ("k8", "v8", "sk", "sv", "state", "weight", "pos", "k_tail", "v_tail")}
    if case["op"] == "step":
        st["state_out"].copy_(st["state"])
        out, wo = st["out"].double(), st["weight_out"].double()
        for b, (n, tl) in enumerate(_rows(case)):
            if n < 0:
                continue
            m = n * BLOCK + tl
            ids = st["table"][b].long()
            st["pos"][b, :, m] = st["state"][b, 2]
            st["k_tail"][b, :, tl], st["v_tail"][b, :, tl] = st["k_new"][b], st["v_new"][b]
            for g in range(hkv):
                pg = ids[g, :n]
                rows = [torch.cat([(st[c][pg].double() * st[s][pg].double()[:, None, None]).view(-1, d), st[t][b, g, :tl + 1].double()])
                        for c, s, t in (("k8", "sk", "k_tail"), ("v8", "sv", "v_tail"))]
                p = torch.softmax(st["q"][b, g * grp:(g + 1) * grp].double() @ rows[0].T * scale, 1)
                out[b, g * grp:(g + 1) * grp] = p @ rows[1]
                wo[b, g, :m + 1] = p.sum(0)
                wo[b, g, :m] += st["weight"][b, g, :m].double()
                if tl == BLOCK - 1:
                    for c, s, t in (("k8", "sk", "k_tail"), ("v8", "sv", "v_tail")):
                        st[c][ids[g, n:n + 1]], st[s][ids[g, n:n + 1]] = _codes64(st[t][b, g:g + 1].double())
            st["state_out"][b, 0], st["state_out"][b, 1] = n + (tl == BLOCK - 1), (tl + 1) % BLOCK
            st["state_out"][b, 2] += 1
        return {n: st[n] for n in ("k8", "v8", "sk", "sv")} | {"out": out, "weight_out": wo} | {
            n: st[n] for n in ("state_out", "pos", "k_tail", "v_tail")}
    for name in ("table", "state", "weight", "pos"):
        st[name + "_out"].copy_(st[name])
    keep = case["keep"]
    for b, (n, tail) in enumerate(_rows(case)):
        if n <= keep:
            continue
        st["state_out"][b, 0] = keep
        body, end = n * BLOCK, keep * BLOCK + tail
        for g in range(hkv):
            row = st["table"][b, g]
            kept = _lexkept(st["weight"][b, g, :body].cpu().numpy(), max(body + tail - case["recent"], body - keep * BLOCK), keep * BLOCK)
            idx = torch.from_numpy(np.concatenate([kept, np.arange(body, body + tail)])).cuda()
            for name in ("weight", "pos"):
                st[name + "_out"][b, g] = 0
                st[name + "_out"][b, g, :end] = st[name][b, g][idx]
            st["table_out"][b, g, :keep] = row[n:n + keep]
            st["table_out"][b, g, keep:keep + n] = row[:n]
            tok = idx[:keep * BLOCK]
            for c, s in (("k8", "sk"), ("v8", "sv")):
                src = row[:n].long()[tok // BLOCK]
                # the survivor's value is fl32(code x scale) by the definition
                x = (st[c][src, tok % BLOCK].double() * st[s][src].double()[:, None]).float().double().view(keep, BLOCK, d)
                dst = row[n:n + keep].long()
                st[c][dst], st[s][dst] = _codes64(x)
    return {n: st[n] for n in ("k8", "v8", "sk", "sv")} | {n + "_out": st[n + "_out"] for n in ("table", "state", "weight", "pos")}
