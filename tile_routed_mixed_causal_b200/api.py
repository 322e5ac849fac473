"""Plans that wire the four ABI calls together with torch-owned buffers.

``PrefillPlan``: quantize_qkv_tiles -> build_tile_lists -> routed_attention_prefill.
``DecodePlan``:  build_tile_lists (decode-cache kind, once) -> routed_attention_decode
per step, over the K/V tiles a PrefillPlan (or quantize_qkv_tiles) produced.
``HybridDecodePlan``: hybrid_select_tokens (once, over the prefix) ->
hybrid_attention_decode per step (token-level hybrid: INT4 tiles plus bf16 selected
and recent tokens).
``HybridPrefillPlan``: quantize_qkv_tiles (K and V INT4 scales) ->
hybrid_select_tokens -> hybrid_attention_prefill.
``EvictingDecodePlan``: attention_weight_sums -> paged_cache_fill (once, over the prompt)
-> paged_attention_decode per step, with paged_cache_evict whenever a row has no room.
``prompt_importance``: attention_weight_sums as the importance of a hybrid selection.
Buffers are allocated once per plan; ``run``/``step`` only enqueue kernels.  The
decode workspace is zero-filled once (the decode's arrival counters need that, and
every step leaves them at zero).
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import _lib as L


class PrefillPlan:
    def __init__(self, shape: L.Shape, policy: L.Policy, keep_v_cache: bool = False,
                 device="cuda"):
        self.shape, self.policy = shape, policy
        fm = L.FMT_Q8 | L.FMT_K8
        if policy.has_int4:
            fm |= L.FMT_Q4X | L.FMT_K4X     # INT4 codes in the tensor-core operand form
        if policy.has_fp8:
            fm |= L.FMT_Q8F | L.FMT_K8F     # FP8 E4M3 codes of the FP8 band
        if keep_v_cache:
            fm |= L.FMT_K4 | L.FMT_V8 | L.FMT_V4
        self.tiles = L.QTiles(shape, fm, device)
        rows, nnz = L.tile_lists_size(shape, policy, L.LISTS_PREFILL)
        self.rows, self.nnz = rows, nnz
        self.row_ptr = torch.zeros(rows + 1, dtype=torch.int32, device=device)
        self.entries = torch.zeros(max(nnz, 4), dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def quantize(self, q, k, v, stream=None):
        L.quantize_qkv_tiles(self.shape, q, k, v, self.tiles, stream)

    def lists(self, stream=None):
        L.build_tile_lists(self.shape, self.policy, L.LISTS_PREFILL, self.row_ptr, self.entries, stream)

    def attend(self, q, k, v, out, lse=None, scale=None, dump_coords=None, dump_out=None,
               stream=None):
        scale = 1.0 / math.sqrt(self.shape.d) if scale is None else scale
        L.routed_attention_prefill(self.shape, self.policy, q, k, v, self.tiles, self.row_ptr,
                                   self.entries, scale, out, lse, dump_coords, dump_out,
                                   self.status, stream)

    def run(self, q, k, v, out, lse=None, scale=None, stream=None):
        """One full prefill pass: quantise, build traversals, fused attention."""
        self.quantize(q, k, v, stream)
        self.lists(stream)
        self.attend(q, k, v, out, lse, scale, stream=stream)


class DecodePlan:
    def __init__(self, shape: L.Shape, policy: L.Policy, cache: L.QTiles, tail_cap: int,
                 device="cuda"):
        self.shape, self.policy, self.cache = shape, policy, cache
        rows, nnz = L.tile_lists_size(shape, policy, L.LISTS_DECODE_CACHE)
        self.row_ptr = torch.zeros(rows + 1, dtype=torch.int32, device=device)
        self.entries = torch.zeros(max(nnz, 4), dtype=torch.int32, device=device)
        self.nnz = nnz
        B, Hkv, d = shape.B, shape.Hkv, shape.d
        self.k_tail = torch.zeros((B, Hkv, tail_cap, d), dtype=torch.bfloat16, device=device)
        self.v_tail = torch.zeros_like(self.k_tail)
        self.tail_len = torch.zeros(B, dtype=torch.int32, device=device)
        nbytes = L.decode_workspace_bytes(B, shape.Hq, Hkv, d)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def build(self, stream=None):
        L.build_tile_lists(self.shape, self.policy, L.LISTS_DECODE_CACHE, self.row_ptr,
                           self.entries, stream)

    def step(self, q, k_new, v_new, out, scale=None, stream=None):
        scale = 1.0 / math.sqrt(self.shape.d) if scale is None else scale
        L.routed_attention_decode(self.shape, self.policy, q, k_new, v_new, self.cache,
                                  self.row_ptr, self.entries, self.k_tail, self.v_tail,
                                  self.tail_len, scale, out, self.workspace, self.status, stream)


class HybridDecodePlan:
    def __init__(self, shape: L.Shape, cache: L.QTiles, frac: float, window: int, tail_cap: int,
                 device="cuda"):
        self.shape, self.cache = shape, cache
        self.hy = L.Hybrid(shape, frac, window, device)
        B, Hkv, d = shape.B, shape.Hkv, shape.d
        self.k_tail = torch.zeros((B, Hkv, tail_cap, d), dtype=torch.bfloat16, device=device)
        self.v_tail = torch.zeros_like(self.k_tail)
        self.tail_len = torch.zeros(B, dtype=torch.int32, device=device)
        nbytes = L.decode_workspace_bytes(B, shape.Hq, Hkv, d)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def select(self, importance, k, v, stream=None):
        L.hybrid_select_tokens(self.shape, importance, self.hy.frac, k, v, self.hy, stream)

    def step(self, q, k_new, v_new, out, scale=None, stream=None):
        scale = 1.0 / math.sqrt(self.shape.d) if scale is None else scale
        L.hybrid_attention_decode(self.shape, self.hy, q, k_new, v_new, self.cache, self.k_tail,
                                  self.v_tail, self.tail_len, scale, out, self.workspace,
                                  self.status, stream)


class HybridPrefillPlan:
    """Causal prefill of the token-level hybrid: keys outside the query's window are read
    from their INT4 tile unless selected; the selection also serves a HybridDecodePlan."""

    def __init__(self, shape: L.Shape, frac: float, window: int, device="cuda"):
        self.shape = shape
        self.tiles = L.QTiles(shape, L.FMT_K4 | L.FMT_V4, device)
        self.hy = L.Hybrid(shape, frac, window, device)
        ntok = int(shape.cu_host[-1])
        self.k_mix = torch.zeros((max(ntok, 1), shape.Hkv, shape.d), dtype=torch.bfloat16,
                                 device=device)
        self.v_mix = torch.zeros_like(self.k_mix)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def prepare(self, k, v, importance, stream=None):
        """Quantise K and V (INT4 scales) and select the bf16 tokens."""
        L.quantize_qkv_tiles(self.shape, None, k, v, self.tiles, stream)
        L.hybrid_select_tokens(self.shape, importance, self.hy.frac, k, v, self.hy, stream)

    def attend(self, q, k, v, out, lse=None, scale=None, stream=None):
        scale = 1.0 / math.sqrt(self.shape.d) if scale is None else scale
        L.hybrid_attention_prefill(self.shape, self.hy, q, k, v, self.tiles, self.k_mix,
                                   self.v_mix, scale, out, lse, self.status, stream)

    def run(self, q, k, v, importance, out, lse=None, scale=None, stream=None):
        self.prepare(k, v, importance, stream)
        self.attend(q, k, v, out, lse, scale, stream)


def _made_on(stream, device):
    """Context whose new tensors belong to the stream that a call is given (None: the current
    one): their memory is neither taken from work still queued on another stream nor handed to
    one before the call's kernels are done."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def prompt_importance(shape: L.Shape, q, k, n_queries: int = 64, lse=None, scale=None, stream=None):
    """Accumulated attention weight of the prompt's keys, float32 [ntok, Hkv]: the importance
    that hybrid_select_tokens and paged_cache_fill take.  n_queries: the last queries of each
    sequence that count (0: all); lse: what a prefill wrote, or None to compute it.  The result
    is made on `stream`; the current stream may use it too, once it has waited for that one."""
    scale = 1.0 / math.sqrt(shape.d) if scale is None else scale
    given = lse is not None
    caller = torch.cuda.current_stream(q.device) if stream is not None and q.is_cuda else None
    with _made_on(stream, q.device):
        weights = torch.empty((shape.ntok, shape.Hkv), dtype=torch.float32, device=q.device)
        if not given:
            lse = torch.empty((shape.Hq, shape.ntok), dtype=torch.float32, device=q.device)
        L.attention_weight_sums(shape, q, k, weights, lse, n_queries=n_queries, softmax_scale=scale,
                                lse_given=given, stream=stream)
    if caller is not None:
        weights.record_stream(caller)   # its memory waits for what the caller's stream does with it
    return weights


class EvictingDecodePlan:
    """Decoding over a bounded INT8 cache: every row keeps at most `keep` pages of its prompt and
    grows to at most `limit` pages.  When a row there has no room for its next page, rows are cut:
    their tokens of least accumulated attention weight go until `keep` pages are left (the last
    `recent` tokens stay).  Cut are all rows of more than `keep` pages, which makes cuts rare, but lets
    what a row keeps depend on the rows beside it; with per_row only those without room, so that
    a row keeps what it would keep alone.

    The plan counts its rows on the host, as step() is called.  A captured step is counted
    once, however often it is replayed: capture paged_cache_evict (its `least` lets the rows' own
    states decide) and paged_attention_decode for that."""

    def __init__(self, shape: L.Shape, keep: int, limit: int, recent: int = 64, n_queries: int = 64,
                 device="cuda", per_row: bool = False):
        if not 1 <= keep < limit:
            raise ValueError(f"need 1 <= keep < limit (got {keep}, {limit})")
        self.shape, self.keep, self.limit = shape, keep, limit
        self.recent, self.n_queries, self.per_row = recent, n_queries, per_row
        # an eviction writes its `keep` pages beside the row's own
        self.cache = L.PagedCache(shape.B, shape.Hq, shape.Hkv, shape.d, limit + keep, device=device)
        self.rows = None        # [pages, tail] of each row, as the device has them

    @property
    def status(self):
        return self.cache.status

    def prefill(self, q, k, v, lse=None, scale=None, stream=None):
        """Weigh the prompt's keys (by the last n_queries queries) and store what stays; the weights,
        made on `stream`."""
        w = prompt_importance(self.shape, q, k, self.n_queries, lse, scale, stream)
        L.paged_cache_fill(self.cache, self.shape, k, v, keep=self.keep, recent=self.recent, weights=w,
                           stream=stream)
        cu = self.shape.cu_host
        lens = [int(b) - int(a) for a, b in zip(cu, cu[1:])]
        self.rows = [[min(t // L.TILE, self.keep), t % L.TILE] for t in lens]
        return w

    def step(self, q, k_new, v_new, out, scale=None, stream=None):
        """One decoded token per row; where one has no room for its page, rows are cut first."""
        if self.rows is None:
            raise RuntimeError("step() needs a prompt: call prefill() first")
        scale = 1.0 / math.sqrt(self.shape.d) if scale is None else scale
        no_room = self.limit * L.TILE + L.TILE - 1     # tokens of such a row
        if any(n * L.TILE + t >= no_room for n, t in self.rows):
            least = no_room if self.per_row else 0
            L.paged_cache_evict(self.cache, keep=self.keep, recent=self.recent, least=least, stream=stream)
            for r in self.rows:
                if r[0] * L.TILE + r[1] >= least:
                    r[0] = min(r[0], self.keep)
        L.paged_attention_decode(self.cache, q, k_new, v_new, out, softmax_scale=scale, stream=stream)
        for r in self.rows:
            if r[0] >= 0:
                r[0], r[1] = r[0] + (r[1] == L.TILE - 1), (r[1] + 1) % L.TILE

    def retire(self, b: int, stream=None):
        """Row b is done: later steps leave it, its output and the other rows' cuts alone."""
        if self.rows is None:
            raise RuntimeError("retire() needs a prompt: call prefill() first")
        with _made_on(stream, self.cache.device):
            self.cache["state"][b, 0] = -1
        self.rows[b][0] = -1
