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
# tensors, what would be misread (a wrong type, an inner stride, a tensor that
# is too short) is refused here, and a return code that is not MLA_OK raises
# MlaError.  A small step's call takes longer on the host than on the GPU, so
# these functions hand plain integers to the library and ask each tensor only
# for what they check.

_ROW_BYTES = {B.MLA_KV_FP8_E4M3: 576, B.MLA_KV_FP8_DS_MLA: 656, B.MLA_KV_NVFP4_DS_MLA: 352,
              B.MLA_KV_FP8_E4M3_PAGE: 576}
_I32, _I64, _F32, _U8, _BF16 = torch.int32, torch.int64, torch.float32, torch.uint8, torch.bfloat16
_FP8 = torch.float8_e4m3fn


def _refuse(what: str):
    raise B.MlaError(B.MLA_EINVAL, what)


def _check(rc: int, what: str) -> None:
    if rc != B.MLA_OK:
        raise B.MlaError(rc, what)


def _flat(x, dtype, n: int, dev: int, what: str) -> int:
    """Address of a contiguous tensor of `dtype` on device `dev` with at least n elements; 0 for None."""
    if x is None:
        return 0
    if x.dtype is not dtype or not x.is_contiguous() or x.numel() < n or x.get_device() != dev:
        _refuse(what)
    return x.data_ptr()


def _stream_of(dev: int, stream, what: str) -> int:
    """The stream's handle; the tensors' device has to be the current one, on which the library launches."""
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(what + ": tensors that are not on the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _query_args(q_latent, q_pe, q_scale_inv, dev: int, what: str):
    """(tokens, heads, the C arguments q_latent .. q_scale_inv)."""
    tokens, heads, width = q_latent.shape
    dtype = q_latent.dtype
    if q_pe.dtype is not dtype or (dtype is not _BF16 if q_scale_inv is None
                                   else dtype is not _U8 and dtype is not _FP8):
        _refuse(what + ": query type")
    lt, lh, l1 = q_latent.stride()
    pt, ph, p1 = q_pe.stride()
    if (width != 512 or q_pe.shape != (tokens, heads, 64) or l1 != 1 or p1 != 1
            or q_latent.get_device() != dev or q_pe.get_device() != dev):
        _refuse(what + ": query shape")
    return tokens, heads, (q_latent.data_ptr(), lt, lh, q_pe.data_ptr(), pt, ph,
                           _flat(q_scale_inv, _F32, 1, dev, what + ": q_scale_inv"))


def _cache_args(cache, layout, k_scale, dev: int, what: str):
    """The C arguments kv_cache .. k_scale."""
    pages, page, row = cache.shape
    if (cache.dtype is not _U8 or row != _ROW_BYTES.get(layout) or not cache.is_contiguous()
            or cache.get_device() != dev):
        _refuse(what + ": cache")
    return (cache.data_ptr(), pages, page, layout,
            _flat(k_scale, _F32, pages if layout == B.MLA_KV_FP8_E4M3_PAGE else 1, dev, what + ": k_scale"))


def _rows2d(x, dtype, dev: int, what: str):
    """(address, entries between rows, rows, columns) of a [rows, columns] tensor with unit inner stride."""
    rows, cols = x.shape
    st, s1 = x.stride()
    if x.dtype is not dtype or (s1 != 1 and cols > 1) or (rows > 1 and st < cols) or x.get_device() != dev:
        _refuse(what)
    return x.data_ptr(), (st if rows > 1 else cols), rows, cols


def tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size, lens_out,
                free_count_out, slot_mapping, token_row, token_len, cu_tokens, flags=None,
                stream=None) -> None:
    """One step's block tables, slot map and causal lengths (``mla_tables_step``).

    ``block_table`` and ``free_pages`` are updated; ``lens_out`` and
    ``free_count_out`` may be ``lens`` and ``free_count`` themselves."""
    what = "tables_step: arrays"
    dev = lens.get_device()
    rows, tokens, pages = lens.numel(), slot_mapping.numel(), free_pages.numel()
    table_rows, width = block_table.shape
    if table_rows != rows:
        _refuse("tables_step: block table")
    _check(B.load().mla_tables_step(
        rows, _flat(new_tokens, _I32, rows, dev, what), _flat(lens, _I32, rows, dev, what),
        _flat(lens_out, _I32, rows, dev, what), _flat(block_table, _I32, 1, dev, what), width,
        _flat(free_pages, _I32, 1, dev, what), _flat(free_count, _I32, 1, dev, what),
        _flat(free_count_out, _I32, 1, dev, what), pages, page_size, tokens,
        _flat(slot_mapping, _I64, 1, dev, what), _flat(token_row, _I32, tokens, dev, what),
        _flat(token_len, _I32, tokens, dev, what), _flat(cu_tokens, _I32, rows + 1, dev, what),
        _flat(flags, _I32, 1, dev, what), _stream_of(dev, stream, "tables_step")), "mla_tables_step")


def blocks_mean(cache, layout, k_scale, block_table, lens_from, lens_to, mean, flags=None,
                stream=None) -> None:
    """Mean keys ``mean`` [pages, 576] of the blocks between two lengths (``mla_blocks_mean``)."""
    dev = cache.get_device()
    args = _cache_args(cache, layout, k_scale, dev, "blocks_mean")
    table, bt_stride, table_rows, _ = _rows2d(block_table, _I32, dev, "blocks_mean: block table")
    rows = lens_to.numel()
    if table_rows < rows:
        _refuse("blocks_mean: block table")
    _check(B.load().mla_blocks_mean(
        *args, table, bt_stride, rows, _flat(lens_from, _I32, rows, dev, "blocks_mean: lengths"),
        _flat(lens_to, _I32, rows, dev, "blocks_mean: lengths"),
        _flat(mean, _BF16, args[1] * 576, dev, "blocks_mean: mean"),
        _flat(flags, _I32, 1, dev, "blocks_mean: flags"), _stream_of(dev, stream, "blocks_mean")),
        "mla_blocks_mean")


def blocks_score(q_latent, q_pe, mean, page_size, block_table, lens, scores, q_scale_inv=None,
                 token_row=None, flags=None, stream=None) -> None:
    """Scores [tokens, blocks] of every block for every query (``mla_blocks_score``)."""
    dev = q_latent.get_device()
    tokens, heads, query = _query_args(q_latent, q_pe, q_scale_inv, dev, "blocks_score")
    table_rows, width = block_table.shape
    out, out_stride, out_rows, out_cols = _rows2d(scores, _F32, dev, "blocks_score: scores")
    if out_rows < tokens or out_cols < width:
        _refuse("blocks_score: scores")
    pages, columns = mean.shape
    if columns != 576:
        _refuse("blocks_score: mean")
    _check(B.load().mla_blocks_score(
        tokens, heads, *query, _flat(mean, _BF16, 1, dev, "blocks_score: mean"), pages, page_size,
        _flat(block_table, _I32, 1, dev, "blocks_score: block table"), width, table_rows,
        _flat(token_row, _I32, tokens, dev, "blocks_score: token_row"),
        _flat(lens, _I32, tokens, dev, "blocks_score: lengths"), out, out_stride,
        _flat(flags, _I32, 1, dev, "blocks_score: flags"), _stream_of(dev, stream, "blocks_score")),
        "mla_blocks_score")


def blocks_select(scores, lens, page_size, keep_first, keep_last, sel, sel_count, stream=None) -> None:
    """The best-scored blocks ``sel`` [tokens, k] of every query (``mla_blocks_select``)."""
    dev = scores.get_device()
    out, out_stride, tokens, k = _rows2d(sel, _I32, dev, "blocks_select: sel")
    sc, sc_stride, sc_rows, blocks = _rows2d(scores, _F32, dev, "blocks_select: scores")
    if sc_rows < tokens:
        _refuse("blocks_select: scores")
    _check(B.load().mla_blocks_select(
        tokens, sc, sc_stride, blocks, _flat(lens, _I32, tokens, dev, "blocks_select: lengths"), page_size,
        keep_first, keep_last, k, out, out_stride,
        _flat(sel_count, _I32, tokens, dev, "blocks_select: sel_count"),
        _stream_of(dev, stream, "blocks_select")), "mla_blocks_select")


class PagedAttention:
    """Latent attention over the paged cache, with its workspace.

    One object serves up to ``max_batch`` tokens of ``heads`` heads; its calls
    must be ordered on one stream."""

    def __init__(self, max_batch: int, heads: int, device="cuda:0"):
        self.handle = None
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
        dev = q_latent.get_device()
        tokens, heads, query = _query_args(q_latent, q_pe, q_scale_inv, dev, "attention")
        paged = _cache_args(cache, layout, k_scale, dev, "attention")
        table, bt_stride, table_rows, _ = _rows2d(block_table, _I32, dev, "attention: block table")
        if heads != self.heads:
            _refuse("attention: heads")
        sel_ptr = sel_stride = 0
        if sel is not None:
            sel_ptr, sel_stride, sel_rows, _ = _rows2d(sel, _I32, dev, "attention: sel")
            if sel_rows < tokens:
                _refuse("attention: sel")
        if out is None:
            out = torch.empty((tokens, heads, 512), dtype=_BF16, device=q_latent.device)
        ot, oh, o1 = out.stride()
        if out.dtype is not _BF16 or out.shape != (tokens, heads, 512) or o1 != 1 or out.get_device() != dev:
            _refuse("attention: out")
        _check(B.load().mla_attn_decode(
            self.handle, tokens, *query, *paged, table, bt_stride, table_rows,
            _flat(token_row, _I32, tokens, dev, "attention: token_row"),
            _flat(lens, _I32, tokens, dev, "attention: lengths"), sel_ptr, sel_stride,
            _flat(sel_count, _I32, tokens, dev, "attention: sel_count"), softmax_scale, out.data_ptr(), ot, oh,
            _flat(lse, _F32, tokens * heads, dev, "attention: lse"), _stream_of(dev, stream, "attention")),
            "mla_attn_decode")
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
