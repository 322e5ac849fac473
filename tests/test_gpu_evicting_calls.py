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
