"""One DSA layer's hot path, stage after stage, on caller-owned buffers.

``LayerBuffers`` allocates every output and workspace once (PyTorch owns the
memory); ``run_layer`` issues the five library calls in the order of the DSA
module page's pipeline (compress -> index_scores -> topk_pools ->
expand_selection -> MLA over the selected rows) on one stream.

``PagedStep`` holds a serving step over a paged latent cache (module
glm5next_dsa, Modules, attend: the paged decode): plan_step gives the step's new
tokens their sequences, positions and cache rows, append_step stores their latent
rows, attend_step attends to all that they see, or select_step and
attend_selected_step to a selection.  Nothing in it reads the GPU back: a step is
captured into a graph once and replayed for the next tokens.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import ops
from .synth import Batch, PagedCache


@dataclass
class LayerBuffers:
    pool_keys: torch.Tensor
    pool_start: torch.Tensor
    pool_valid: torch.Tensor
    n_pools: torch.Tensor
    scores: torch.Tensor
    pool_ids: torch.Tensor
    token_ids: torch.Tensor
    out: torch.Tensor
    lse: torch.Tensor
    ws_topk: torch.Tensor
    ws_select: torch.Tensor
    ws_mla: torch.Tensor | None
    status: torch.Tensor

    @staticmethod
    def alloc(bt: Batch, device=None) -> "LayerBuffers":
        dev = device or bt.k.device
        g = bt.geo
        total_cap = int(bt.cu_pool_cap[-1].item())
        Q = bt.Q
        ws_t = ops.topk_workspace_bytes(Q, bt.P_ld, g.select_k)
        ws_s = ops.select_workspace_bytes(Q, bt.P_ld, g.select_k)
        tag = ops.DSA_BF16 if g.dtype == "bf16" else ops.DSA_F32
        ws_m = ops.mla_workspace_bytes(Q, g.Hm, g.L, g.out_width, tag)
        return LayerBuffers(
            pool_keys=torch.zeros(max(total_cap, 1), g.D, dtype=bt.k.dtype, device=dev),
            pool_start=torch.full((max(total_cap, 1),), -1, dtype=torch.int32, device=dev),
            pool_valid=torch.zeros(max(total_cap, 1), dtype=torch.uint8, device=dev),
            n_pools=torch.zeros(bt.B, dtype=torch.int32, device=dev),
            scores=torch.empty(Q, bt.P_ld, dtype=torch.float32, device=dev),
            pool_ids=torch.empty(Q, g.select_k, dtype=torch.int32, device=dev),
            token_ids=torch.empty(Q, g.out_width, dtype=torch.int32, device=dev),
            out=torch.empty(Q, g.Hm, g.L, dtype=bt.q_lat.dtype, device=dev),
            lse=torch.empty(Q, g.Hm, dtype=torch.float32, device=dev),
            ws_topk=torch.empty(max(ws_t, 16), dtype=torch.uint8, device=dev),
            ws_select=torch.zeros(max(ws_s, 16), dtype=torch.uint8, device=dev),
            ws_mla=torch.empty(ws_m, dtype=torch.uint8, device=dev) if ws_m else None,
            status=torch.zeros(1, dtype=torch.int32, device=dev))


def compress(bt: Batch, buf: LayerBuffers, pool_begin=None, max_pools=None, stream=None):
    if max_pools is None:
        max_pools = bt.P_ld
    ops.dsa_kpool_compress(bt.k, bt.gate, bt.valid, bt.ape, bt.ln_gamma, bt.ln_beta, bt.geo.ln_eps,
                           bt.cu_seqlens, bt.cu_pool_cap, pool_begin, bt.geo.kpool, max_pools,
                           buf.pool_keys, buf.pool_start, buf.pool_valid, buf.n_pools, buf.status,
                           stream)


def select_stages(bt: Batch, buf: LayerBuffers, stream=None):
    """index_scores -> topk_pools -> expand_selection as three separate calls."""
    g = bt.geo
    ops.dsa_index_scores(bt.q, bt.weights, bt.scale, buf.pool_keys, buf.pool_start,
                         buf.pool_valid, buf.n_pools, bt.cu_pool_cap, bt.q_seq, bt.q_pos,
                         g.kpool, buf.scores, buf.status, stream)
    ops.dsa_topk_pools(buf.scores, g.select_k, buf.pool_ids, buf.ws_topk, stream)
    ops.dsa_expand_selection(buf.pool_ids, buf.pool_start, bt.cu_pool_cap, bt.q_seq, g.kpool,
                             buf.token_ids, buf.status, stream)


def select(bt: Batch, buf: LayerBuffers, stream=None):
    """The fused select call (same outputs as select_stages)."""
    ops.dsa_select(bt.q, bt.weights, bt.scale, buf.pool_keys, buf.pool_start, buf.pool_valid,
                   buf.n_pools, bt.cu_pool_cap, bt.q_seq, bt.q_pos, bt.geo.kpool, buf.scores,
                   buf.pool_ids, buf.token_ids, buf.ws_select, buf.status, stream)


def attend(bt: Batch, buf: LayerBuffers, stream=None):
    ops.dsa_mla_selected_decode(bt.q_lat, bt.kv, bt.cu_seqlens, bt.q_seq, buf.token_ids,
                                bt.sm_scale, buf.out, buf.lse, buf.ws_mla, buf.status, stream)


def decode_layer(bt: Batch, buf: LayerBuffers, pool_begin=None, max_pools=None, stream=None):
    """compress -> select -> attend as the single fused call (same outputs as
    run_layer)."""
    if max_pools is None:
        max_pools = bt.P_ld
    ops.dsa_decode_layer(bt.k, bt.gate, bt.valid, bt.ape, bt.ln_gamma, bt.ln_beta, bt.geo.ln_eps,
                         bt.cu_seqlens, pool_begin, max_pools, buf.pool_keys, buf.pool_start,
                         buf.pool_valid, buf.n_pools, bt.cu_pool_cap, bt.q, bt.weights, bt.scale,
                         bt.q_seq, bt.q_pos, bt.q_lat, bt.kv, bt.sm_scale, bt.geo.kpool,
                         buf.scores, buf.pool_ids, buf.token_ids, buf.out, buf.lse,
                         buf.ws_select, buf.ws_mla, buf.status, stream)


def run_layer(bt: Batch, buf: LayerBuffers, pool_begin=None, max_pools=None, stream=None,
              fused=True):
    compress(bt, buf, pool_begin, max_pools, stream)
    (select if fused else select_stages)(bt, buf, stream)
    attend(bt, buf, stream)


@dataclass
class ProjectionBuffers:
    """Outputs and workspace of dsa_indexer_project for one layer."""
    k: torch.Tensor          # [rows, D] bf16 (rows = T, or the cache rows kv_rows points into)
    gate: torch.Tensor       # [rows, D] bf16
    weights: torch.Tensor    # [T, H] fp32
    q: torch.Tensor          # [T, H, D] bf16
    q_nope: torch.Tensor     # [T, Hm, nope] bf16
    q_lat: torch.Tensor      # [T, Hm, L] bf16
    ws: torch.Tensor | None  # counters zeroed here, left zero by every call
    status: torch.Tensor

    @staticmethod
    def alloc(pi, rows=None, device=None) -> "ProjectionBuffers":
        dev = device or pi.x.device
        T, hidden = pi.x.shape
        bf = torch.bfloat16
        rows = T if rows is None else rows
        ws = ops.indexer_project_workspace_bytes(T, hidden, pi.cq.shape[1], pi.H, pi.D, pi.Hm,
                                                 pi.nope, pi.L)
        return ProjectionBuffers(
            k=torch.zeros(rows, pi.D, dtype=bf, device=dev),
            gate=torch.zeros(rows, pi.D, dtype=bf, device=dev),
            weights=torch.empty(T, pi.H, dtype=torch.float32, device=dev),
            q=torch.empty(T, pi.H, pi.D, dtype=bf, device=dev),
            q_nope=torch.empty(T, pi.Hm, pi.nope, dtype=bf, device=dev),
            q_lat=torch.empty(T, pi.Hm, pi.L, dtype=bf, device=dev),
            ws=torch.zeros(ws, dtype=torch.uint8, device=dev) if ws else None,
            status=torch.zeros(1, dtype=torch.int32, device=dev))


def project(pi, buf: ProjectionBuffers, weights_scale: float, kv_rows=None, stream=None):
    """The indexer projections of one layer: k, gate, weights, q, q_nope, q_lat."""
    ops.dsa_indexer_project(pi.x, pi.w_kgw, pi.cq, pi.w_q, pi.w_uk_t, weights_scale, buf.k,
                            buf.gate, buf.weights, buf.q, buf.q_nope, buf.q_lat, buf.ws,
                            kv_rows, buf.status, stream)


@dataclass
class PagedStep:
    """Buffers of a serving step of up to T new tokens over a ``PagedCache`` whose pages come
    from one free list; every layer of a model shares the plan, its cache rows and pages."""
    free_pages: torch.Tensor   # [n_free] int32 pages, taken from free_begin on
    free_begin: torch.Tensor   # [1] int32
    cu_new: torch.Tensor       # [B + 1] int32: the plan's token axis
    q_seq: torch.Tensor        # [T] int32
    q_pos: torch.Tensor
    kv_rows: torch.Tensor
    key_rows: torch.Tensor
    out: torch.Tensor          # [T, Hm, L]
    lse: torch.Tensor          # [T, Hm] fp32
    ws: torch.Tensor | None
    status: torch.Tensor
    scores: torch.Tensor | None = None        # a selection's (alloc with its batch)
    pool_ids: torch.Tensor | None = None
    token_ids: torch.Tensor | None = None     # [T, out_width] int32
    ws_select: torch.Tensor | None = None
    ws_selected: torch.Tensor | None = None

    @staticmethod
    def alloc(cache: PagedCache, free_pages, T: int, Hm: int, dtype=torch.bfloat16,
              bt: Batch | None = None) -> "PagedStep":
        dev, L = cache.pages.device, cache.pages.shape[1]
        B = cache.seq_lens.numel()
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
        out = torch.zeros(T, Hm, L, dtype=dtype, device=dev)
        ws = ops.mla_paged_chunk_workspace_bytes(out, cache.pages)
        step = PagedStep(
            free_pages=free_pages, free_begin=i32(1), cu_new=i32(B + 1), q_seq=i32(T),
            q_pos=i32(T), kv_rows=i32(T), key_rows=i32(T), out=out,
            lse=torch.zeros(T, Hm, dtype=torch.float32, device=dev),
            ws=torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None, status=i32(1))
        if bt is not None:
            g = bt.geo
            ws_s = ops.select_workspace_bytes(T, bt.P_ld, g.select_k)
            ws_m = ops.mla_paged_workspace_bytes(out, cache.pages, g.out_width)
            step.scores = torch.empty(T, bt.P_ld, dtype=torch.float32, device=dev)
            step.pool_ids = torch.empty(T, g.select_k, dtype=torch.int32, device=dev)
            step.token_ids = torch.empty(T, g.out_width, dtype=torch.int32, device=dev)
            step.ws_select = torch.zeros(max(ws_s, 16), dtype=torch.uint8, device=dev)
            step.ws_selected = torch.empty(max(ws_m, 16), dtype=torch.uint8, device=dev)
        return step


def plan_step(cache: PagedCache, step: PagedStep, new_lens, row_base=None, stream=None):
    """The step of ``new_lens`` [B] tokens: lengths, table and free list move on in place."""
    ops.dsa_paged_plan(cache.seq_lens, new_lens, step.free_pages, step.free_begin,
                       cache.pages.shape[0] // cache.page_size, cache.page_size,
                       cache.block_table, cache.seq_lens, step.cu_new, step.q_seq, step.q_pos,
                       step.kv_rows, step.free_begin, row_base,
                       None if row_base is None else step.key_rows, step.status, stream)


def append_step(cache: PagedCache, step: PagedStep, kv_new, stream=None):
    """Store the step's latent rows ``kv_new`` [T, L] in one layer's cache."""
    ops.dsa_paged_append(kv_new, step.kv_rows, cache.pages, cache.row_scale, step.status, stream)


def attend_step(cache: PagedCache, step: PagedStep, q_lat, sm_scale, window=0, sinks=0,
                stream=None):
    """Dense attention of the step's tokens (``q_lat`` [T, Hm, L]) into ``step.out``, ``lse``."""
    ops.dsa_mla_paged_chunk(q_lat, cache.pages, cache.row_scale, cache.block_table,
                            cache.seq_lens, cache.page_size, step.cu_new, window, sinks, sm_scale,
                            step.out, step.lse, step.ws, step.status, stream)


def select_step(bt: Batch, buf: LayerBuffers, step: PagedStep, q, weights, stream=None):
    """``step.token_ids``: what the step's tokens select among the pools of ``buf`` (``q``
    [T, H, D], ``weights`` [T, H]); rows behind the last token select nothing."""
    ops.dsa_select(q, weights, bt.scale, buf.pool_keys, buf.pool_start, buf.pool_valid,
                   buf.n_pools, bt.cu_pool_cap, step.q_seq, step.q_pos, bt.geo.kpool, step.scores,
                   step.pool_ids, step.token_ids, step.ws_select, step.status, stream)


def attend_selected_step(cache: PagedCache, step: PagedStep, q_lat, sm_scale, stream=None):
    """Attention of the step's tokens over ``step.token_ids`` into ``step.out``, ``lse``."""
    ops.dsa_mla_paged_decode(q_lat, cache.pages, cache.row_scale, cache.block_table,
                             cache.seq_lens, cache.page_size, step.q_seq, step.token_ids, sm_scale,
                             step.out, step.lse, step.ws_selected, step.status, stream)
