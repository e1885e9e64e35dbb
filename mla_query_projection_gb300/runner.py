"""Torch-side plumbing around the C ABI: device buffers for one decode step.

PyTorch only allocates memory and provides the stream; the decode itself is
one ``mla_query_decode`` call into the CUDA library.
"""

from __future__ import annotations

import contextlib
import ctypes

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
        # one scale, or one for each page (MLA_KV_FP8_E4M3_PAGE)
        self.k_scale = torch.tensor(np.atleast_1d(inp["k_scale"]), dtype=torch.float32, device=dev)
        self.eps = float(inp["eps"])
        self.q_latent = torch.empty((Bn, H, 512), dtype=torch.bfloat16, device=dev)
        self.q_pe = torch.empty((Bn, H, 64), dtype=torch.bfloat16, device=dev)
        self.q_c = torch.empty((Bn, 1536), dtype=torch.bfloat16, device=dev) if q_c else None
        self.handle = B.mla_query_create(H, self.w_qb, self.w_uk, self.gamma_q, self.gamma_kv, self.eps)

    def decode(self, stream=None, batch=None) -> int:
        if self.layout == B.MLA_KV_FP8_E4M3_PAGE and (
                self.k_scale.numel() < self.num_pages or not self.k_scale.is_contiguous()):
            return B.MLA_EINVAL  # the kernel would read behind the scales
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
# Thin calls over the C ABI for torch tensors (csrc/torch/tensor_calls.cpp):
# sizes and strides come from the tensors; what would be misread (a wrong type,
# an inner stride, a tensor that is too short or off the current device) is
# refused before anything is launched, and raises MlaError as a return code that
# is not MLA_OK does.  `stream` is a torch stream, a handle, or None for the
# current one.

_calls = None


def _native():
    """The module that checks the tensors and calls the library, bound to the loaded build."""
    global _calls
    if _calls is None:
        lib = B.load()
        try:
            from . import _tensor_calls
        except ImportError as e:
            raise RuntimeError("mla_query_projection_gb300/_tensor_calls.so is not built: build it with "
                               "`python -m mla_query_projection_gb300.build`") from e
        _tensor_calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.mla_tables_step, lib.mla_blocks_mean_cols, lib.mla_blocks_score, lib.mla_blocks_select,
            lib.mla_attn_decode_cols)))
        _calls = _tensor_calls
    return _calls


def _refuse(wrong, what: str):
    """What a call gave back instead of None: what is wrong with its tensors, or a return code."""
    if isinstance(wrong, str):
        raise B.MlaError(B.MLA_EINVAL, f"{what}: {wrong}")
    raise B.MlaError(wrong, what)


def tables_step(new_tokens, lens, block_table, free_pages, free_count, page_size, lens_out,
                free_count_out, slot_mapping, token_row, token_len, cu_tokens, flags=None,
                stream=None) -> None:
    """One step's block tables, slot map and causal lengths (``mla_tables_step``).

    ``block_table`` and ``free_pages`` are updated; ``lens_out`` and
    ``free_count_out`` may be ``lens`` and ``free_count`` themselves."""
    wrong = (_calls or _native()).tables_step(
        new_tokens, lens, block_table, free_pages, free_count, page_size, lens_out, free_count_out,
        slot_mapping, token_row, token_len, cu_tokens, flags, stream)
    if wrong is not None:
        _refuse(wrong, "mla_tables_step")


def blocks_mean(cache, layout, k_scale, block_table, lens_from, lens_to, mean, flags=None,
                stream=None) -> None:
    """Mean keys ``mean`` [pages, 576] of the blocks between two lengths (``mla_blocks_mean``)."""
    wrong = (_calls or _native()).blocks_mean(cache, layout, k_scale, block_table, lens_from, lens_to, mean,
                                              flags, stream)
    if wrong is not None:
        _refuse(wrong, "mla_blocks_mean")


def blocks_score(q_latent, q_pe, mean, page_size, block_table, lens, scores, q_scale_inv=None,
                 token_row=None, flags=None, stream=None) -> None:
    """Scores [tokens, blocks] of every block for every query (``mla_blocks_score``)."""
    wrong = (_calls or _native()).blocks_score(q_latent, q_pe, mean, page_size, block_table, lens, scores,
                                               q_scale_inv, token_row, flags, stream)
    if wrong is not None:
        _refuse(wrong, "mla_blocks_score")


def blocks_select(scores, lens, page_size, keep_first, keep_last, sel, sel_count, stream=None) -> None:
    """The best-scored blocks ``sel`` [tokens, k] of every query (``mla_blocks_select``)."""
    wrong = (_calls or _native()).blocks_select(scores, lens, page_size, keep_first, keep_last, sel, sel_count,
                                                stream)
    if wrong is not None:
        _refuse(wrong, "mla_blocks_select")


def _allocating_on(stream, device):
    """A context whose allocations belong to the stream that a call is given, in any of its
    forms: memory of another stream may still be in use there, or be handed out there again,
    while this call's kernels run."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = getattr(stream, "cuda_stream", stream)
        if not isinstance(handle, int):  # None: the current one (anything else is refused by the call)
            return contextlib.nullcontext()
        # (0 and 1: the legacy default stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


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
        be strided (views of gathered rows), and so may ``block_table`` and
        ``sel`` (the first columns of wider tables: only those count).
        ``out`` BF16 [tokens, heads, 512] is allocated, as memory of the
        call's stream, where it is not given; ``lse`` FP32 [tokens, heads] is
        written where it is."""
        if out is None and isinstance(q_latent, torch.Tensor) and q_latent.is_cuda:
            with _allocating_on(stream, q_latent.device):
                out = torch.empty((*q_latent.shape[:2], 512), dtype=torch.bfloat16, device=q_latent.device)
        wrong = (_calls or _native()).attn_decode(
            self.handle, self.heads, q_latent, q_pe, cache, layout, block_table, lens, softmax_scale, k_scale,
            q_scale_inv, token_row, sel, sel_count, out, lse, stream)
        if wrong is not None:
            _refuse(wrong, "mla_attn_decode")
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
