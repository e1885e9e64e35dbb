"""Torch-side plumbing around the C ABI: device buffers for one decode step.

PyTorch only allocates memory and provides the stream; the decode itself is
one ``mla_query_decode`` call into the CUDA library.
"""

from __future__ import annotations

import numpy as np
import torch

from . import binding as B


def bf16_tensor(bits: np.ndarray, device) -> torch.Tensor:
    """uint16 BF16 bit patterns -> torch.bfloat16 tensor on `device`."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.view(torch.bfloat16).to(device)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


class DecodeStep:
    """Device copies of one workload's inputs and outputs plus a handle.

    ``fused_row=True`` packs q_a | kv_c | k_pe into one [B, 2112] row (strided
    inputs, the layout of a fused qkv activation).  ``hidden=True`` makes that
    row on the device instead: every ``decode`` first runs the qkv_a
    down-projection of ``inp["hidden"]`` through ``inp["w_qkv_a"]`` into it."""

    def __init__(self, inp: dict, device="cuda:0", fused_row: bool = False, q_c: bool = True,
                 weights: dict | None = None, hidden: bool = False):
        self.device = torch.device(device)
        dev = self.device
        self.batch = int(inp["q_a"].shape[0])
        self.heads = int(inp["w_uk"].shape[0])
        self.layout = int(inp["layout"])
        wsrc = weights if weights is not None else inp
        if weights is not None and isinstance(weights.get("w_qb"), torch.Tensor):
            self.w_qb, self.w_uk = weights["w_qb"], weights["w_uk"]
            self.gamma_q, self.gamma_kv = weights["gamma_q"], weights["gamma_kv"]
        else:
            self.w_qb = bf16_tensor(wsrc["w_qb"], dev)
            self.w_uk = bf16_tensor(wsrc["w_uk"], dev)
            self.gamma_q = bf16_tensor(wsrc["gamma_q"], dev)
            self.gamma_kv = bf16_tensor(wsrc["gamma_kv"], dev)
        Bn, H = self.batch, self.heads
        self.qkv_a = None
        if hidden:
            self.w_qkv_a = bf16_tensor(inp["w_qkv_a"], dev)
            self.hidden = bf16_tensor(inp["hidden"], dev)
            n, k = self.w_qkv_a.shape
            self.qkv_a = B.mla_qkv_a_create(n, k, self.w_qkv_a)
            fused_row = True
        if fused_row:
            row = np.zeros((Bn, 2112), dtype=np.uint16)
            row[:, :1536] = inp["q_a"]
            row[:, 1536:2048] = inp["kv_c"]
            row[:, 2048:] = inp["k_pe"]
            self.row = bf16_tensor(row, dev)
            self.q_a, self.kv_c, self.k_pe = self.row[:, :1536], self.row[:, 1536:2048], self.row[:, 2048:]
            self.strides = (2112, 2112, 2112)
        else:
            self.q_a = bf16_tensor(inp["q_a"], dev)
            self.kv_c = bf16_tensor(inp["kv_c"], dev)
            self.k_pe = bf16_tensor(inp["k_pe"], dev)
            self.strides = (0, 0, 0)
        self.slots = torch.from_numpy(np.asarray(inp["slots"], dtype=np.int64)).to(dev)
        self.cache = torch.from_numpy(np.ascontiguousarray(inp["cache"])).to(dev)
        self.num_pages, self.page_size = int(self.cache.shape[0]), int(self.cache.shape[1])
        self.k_scale = torch.tensor([inp["k_scale"]], dtype=torch.float32, device=dev)
        self.eps = float(inp["eps"])
        self.q_latent = torch.empty((Bn, H, 512), dtype=torch.bfloat16, device=dev)
        self.q_pe = torch.empty((Bn, H, 64), dtype=torch.bfloat16, device=dev)
        self.q_c = torch.empty((Bn, 1536), dtype=torch.bfloat16, device=dev) if q_c else None
        self.handle = B.mla_query_create(H, self.w_qb, self.w_uk, self.gamma_q, self.gamma_kv, self.eps)

    def decode(self, stream=None, batch=None) -> int:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if self.qkv_a is not None:
            rc = B.mla_qkv_a_run(self.qkv_a, self.batch if batch is None else batch, self.hidden, 0,
                                 self.row, 2112, s)
            if rc != B.MLA_OK:
                return rc
        return B.mla_query_decode(
            self.handle, self.batch if batch is None else batch,
            self.q_a, self.strides[0], self.kv_c, self.strides[1], self.k_pe, self.strides[2],
            self.slots, self.cache, self.num_pages, self.page_size, self.layout, self.k_scale,
            self.q_latent, self.q_pe, self.q_c, s,
        )

    def set_path(self, path: int) -> int:
        return B.mla_query_set_path(self.handle, path)

    def error_flags(self) -> int:
        return B.mla_query_get_error(self.handle, torch.cuda.current_stream(self.device))

    def results(self) -> dict:
        torch.cuda.synchronize(self.device)
        out = {
            "q_latent": bf16_bits(self.q_latent),
            "q_pe": bf16_bits(self.q_pe),
            "cache": self.cache.cpu().numpy(),
        }
        if self.q_c is not None:
            out["q_c"] = bf16_bits(self.q_c)
        if self.qkv_a is not None:
            out["qkv_row"] = bf16_bits(self.row)
        return out

    def close(self):
        if self.handle:
            torch.cuda.synchronize(self.device)
            B.mla_query_destroy(self.handle)
            self.handle = None
        if self.qkv_a is not None:
            B.mla_qkv_a_destroy(self.qkv_a)
            self.qkv_a = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- the cache side of the step -------------------------------------------
#
# Thin calls over the C ABI for torch tensors: sizes and strides come from the
# tensors, what would be misread (a wrong type, an inner stride) is refused
# here, and a return code that is not MLA_OK raises MlaError.

_ROW_BYTES = {B.MLA_KV_FP8_E4M3: 576, B.MLA_KV_FP8_DS_MLA: 656, B.MLA_KV_NVFP4_DS_MLA: 352,
              B.MLA_KV_FP8_E4M3_PAGE: 576}


def _check(rc: int, what: str) -> None:
    if rc != B.MLA_OK:
        raise B.MlaError(rc, what)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise B.MlaError(B.MLA_EINVAL, what)


def _flat(x, dtype, n: int | None, what: str) -> None:
    """`x` is None or a contiguous tensor of `dtype` with at least n elements."""
    if x is not None:
        _need(x.dtype == dtype and x.is_contiguous() and (n is None or x.numel() >= n), what)


def _stream_of(t: torch.Tensor, stream):
    return torch.cuda.current_stream(t.device) if stream is None else stream


def _queries(q_latent, q_pe, q_scale_inv, what: str):
    tokens, heads = q_latent.shape[0], q_latent.shape[1]
    dtypes = (torch.bfloat16,) if q_scale_inv is None else (torch.uint8, torch.float8_e4m3fn)
    _need(q_latent.dtype in dtypes and q_pe.dtype in dtypes, what + ": query type")
    _need(q_latent.shape[2] == 512 and tuple(q_pe.shape) == (tokens, heads, 64)
          and q_latent.stride(2) == 1 and q_pe.stride(2) == 1, what + ": query shape")
    _flat(q_scale_inv, torch.float32, 1, what + ": q_scale_inv")
    return tokens, heads


def _paged(cache, layout, k_scale, table, what: str):
    _need(cache.dtype == torch.uint8 and cache.is_contiguous() and cache.dim() == 3
          and cache.shape[2] == _ROW_BYTES.get(layout), what + ": cache")
    _flat(k_scale, torch.float32, cache.shape[0] if layout == B.MLA_KV_FP8_E4M3_PAGE else 1,
          what + ": k_scale")
    _need(table.dtype == torch.int32 and table.dim() == 2 and table.stride(1) == 1
          and (table.shape[0] == 1 or table.stride(0) >= table.shape[1]), what + ": block table")


def _wide(table: torch.Tensor) -> int:
    """Entries between two rows of a [rows][blocks] table."""
    return table.stride(0) if table.shape[0] > 1 else table.shape[1]


def tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size, lens_out,
                free_count_out, slot_mapping, token_row, token_len, cu_tokens, flags=None,
                stream=None) -> None:
    """One step's block tables, slot map and causal lengths (``mla_tables_step``).

    ``block_table`` and ``free_pages`` are updated; ``lens_out`` and
    ``free_count_out`` may be ``lens`` and ``free_count`` themselves."""
    rows, tokens, i32 = lens.shape[0], slot_mapping.shape[0], torch.int32
    for x, n in ((new_tokens, rows), (lens, rows), (lens_out, rows), (free_pages, None),
                 (free_count, 1), (free_count_out, 1), (token_row, tokens), (token_len, tokens),
                 (cu_tokens, rows + 1), (block_table, None), (flags, 1)):
        _flat(x, i32, n, "tables_step: int32 arrays")
    _flat(slot_mapping, torch.int64, tokens, "tables_step: slot_mapping")
    _need(block_table.dim() == 2 and block_table.shape[0] == rows, "tables_step: block table")
    _check(B.mla_tables_step(
        rows, new_tokens, lens, lens_out, block_table, block_table.shape[1], free_pages, free_count,
        free_count_out, free_pages.shape[0], page_size, tokens, slot_mapping, token_row, token_len,
        cu_tokens, flags, _stream_of(lens, stream)), "mla_tables_step")


def blocks_mean(cache, layout, k_scale, block_table, lens_from, lens_to, mean, flags=None,
                stream=None) -> None:
    """Mean keys ``mean`` [pages, 576] of the blocks between two lengths (``mla_blocks_mean``)."""
    _paged(cache, layout, k_scale, block_table, "blocks_mean")
    rows = lens_to.shape[0]
    _flat(lens_from, torch.int32, rows, "blocks_mean: lengths")
    _flat(lens_to, torch.int32, rows, "blocks_mean: lengths")
    _flat(flags, torch.int32, 1, "blocks_mean: flags")
    _flat(mean, torch.bfloat16, cache.shape[0] * 576, "blocks_mean: mean")
    _need(block_table.shape[0] >= rows, "blocks_mean: block table")
    _check(B.mla_blocks_mean(
        cache, cache.shape[0], cache.shape[1], layout, k_scale, block_table, _wide(block_table), rows,
        lens_from, lens_to, mean, flags, _stream_of(cache, stream)), "mla_blocks_mean")


def blocks_score(q_latent, q_pe, mean, page_size, block_table, lens, scores, q_scale_inv=None,
                 token_row=None, flags=None, stream=None) -> None:
    """Scores [tokens, blocks] of every block for every query (``mla_blocks_score``)."""
    tokens, heads = _queries(q_latent, q_pe, q_scale_inv, "blocks_score")
    _flat(mean, torch.bfloat16, None, "blocks_score: mean")
    _flat(lens, torch.int32, tokens, "blocks_score: lengths")
    _flat(token_row, torch.int32, tokens, "blocks_score: token_row")
    _flat(flags, torch.int32, 1, "blocks_score: flags")
    _need(block_table.dtype == torch.int32 and block_table.is_contiguous()
          and scores.dtype == torch.float32 and scores.stride(1) == 1 and scores.shape[0] >= tokens
          and scores.shape[1] >= block_table.shape[1], "blocks_score: block table or scores")
    _check(B.mla_blocks_score(
        tokens, heads, q_latent, q_latent.stride(0), q_latent.stride(1), q_pe, q_pe.stride(0),
        q_pe.stride(1), q_scale_inv, mean, mean.shape[0], page_size, block_table,
        block_table.shape[1], block_table.shape[0], token_row, lens, scores, _wide(scores), flags,
        _stream_of(q_latent, stream)), "mla_blocks_score")


def blocks_select(scores, lens, page_size, keep_first, keep_last, sel, sel_count, stream=None) -> None:
    """The best-scored blocks ``sel`` [tokens, k] of every query (``mla_blocks_select``)."""
    tokens, k = sel.shape
    _need(scores.dtype == torch.float32 and scores.stride(1) == 1 and scores.shape[0] >= tokens,
          "blocks_select: scores")
    _need(sel.dtype == torch.int32 and sel.stride(1) == 1, "blocks_select: sel")
    _flat(lens, torch.int32, tokens, "blocks_select: lengths")
    _flat(sel_count, torch.int32, tokens, "blocks_select: sel_count")
    _check(B.mla_blocks_select(
        tokens, scores, _wide(scores), scores.shape[1], lens, page_size, keep_first, keep_last, k,
        sel, _wide(sel), sel_count, _stream_of(scores, stream)), "mla_blocks_select")


class PagedAttention:
    """Latent attention over the paged cache, with its workspace.

    One object serves up to ``max_batch`` tokens of ``heads`` heads; its calls
    must be ordered on one stream."""

    def __init__(self, max_batch: int, heads: int, device="cuda:0"):
        self.device = torch.device(device)
        self.heads = heads
        with torch.cuda.device(self.device):
            self.handle = B.mla_attn_create(max_batch, heads)

    def decode(self, q_latent, q_pe, cache, layout, block_table, lens, softmax_scale, k_scale=None,
               q_scale_inv=None, token_row=None, sel=None, sel_count=None, out=None, lse=None,
               stream=None):
        """Attention of the query tokens (``mla_attn_decode``); returns ``(out, lse)``.

        ``q_latent`` [tokens, heads, 512] and ``q_pe`` [tokens, heads, 64] may
        be strided (views of gathered rows); ``out`` BF16 [tokens, heads, 512]
        is allocated where it is not given, ``lse`` FP32 [tokens, heads] is
        written where it is."""
        tokens, heads = _queries(q_latent, q_pe, q_scale_inv, "attention")
        _paged(cache, layout, k_scale, block_table, "attention")
        _need(heads == self.heads, "attention: heads")
        _flat(lens, torch.int32, tokens, "attention: lengths")
        _flat(token_row, torch.int32, tokens, "attention: token_row")
        _flat(sel_count, torch.int32, tokens, "attention: sel_count")
        _flat(lse, torch.float32, tokens * heads, "attention: lse")
        sel_stride = 0
        if sel is not None:
            _need(sel.dtype == torch.int32 and sel.stride(1) == 1 and sel.shape[0] >= tokens,
                  "attention: sel")
            sel_stride = _wide(sel)
        if out is None:
            out = torch.empty((tokens, heads, 512), dtype=torch.bfloat16, device=q_latent.device)
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (tokens, heads, 512)
              and out.stride(2) == 1, "attention: out")
        _check(B.mla_attn_decode(
            self.handle, tokens, q_latent, q_latent.stride(0), q_latent.stride(1), q_pe,
            q_pe.stride(0), q_pe.stride(1), q_scale_inv, cache, cache.shape[0], cache.shape[1], layout,
            k_scale, block_table, _wide(block_table), block_table.shape[0], token_row, lens, sel,
            sel_stride, sel_count, softmax_scale, out, out.stride(0), out.stride(1), lse,
            _stream_of(q_latent, stream)), "mla_attn_decode")
        return out, lse

    def error_flags(self) -> int:
        return B.mla_attn_get_error(self.handle, torch.cuda.current_stream(self.device))

    def close(self):
        if self.handle:
            torch.cuda.synchronize(self.device)
            B.mla_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
