"""Host checks of the cache-side entry points: what the documentation rules out
is refused with MLA_EINVAL before anything reaches the device (CPU only)."""

import ctypes
import os

import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mla_query_projection_gb300 import build

        build.build()
    return B.load()


P = 4096  # an aligned address that no call may follow

TABLES = dict(rows=4, new_tokens=P, lens=P, lens_out=P, block_table=P, bt_stride=8, free_pages=P,
              free_count=P, free_count_out=P, num_pages=16, page_size=64, max_tokens=4,
              slot_mapping=P, token_row=P, token_len=P, cu_tokens=P, device_flags=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(rows=0), dict(rows=B.MLA_MAX_TABLE_ROWS + 1), dict(bt_stride=0), dict(num_pages=0),
    dict(num_pages=1 << 31), dict(page_size=0), dict(max_tokens=0), dict(new_tokens=None),
    dict(lens=None), dict(lens_out=None), dict(block_table=None), dict(free_pages=None),
    dict(free_count=None), dict(free_count_out=None), dict(slot_mapping=None),
    dict(token_row=None), dict(token_len=None), dict(cu_tokens=None), dict(lens=P + 2),
    dict(slot_mapping=P + 4), dict(device_flags=P + 1),
])
def test_tables_step_refuses(change):
    assert B.mla_tables_step(**{**TABLES, **change}) == B.MLA_EINVAL


MEAN = dict(kv_cache=P, num_pages=16, page_size=64, layout=0, k_scale=P, block_table=P, bt_stride=8,
            rows=2, lens_from=P, lens_to=P, mean=P, device_flags=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(kv_cache=None), dict(kv_cache=P + 8), dict(num_pages=0), dict(page_size=0), dict(layout=4),
    dict(layout=-1), dict(k_scale=None), dict(layout=3, k_scale=None), dict(block_table=None),
    dict(bt_stride=0), dict(rows=0), dict(rows=B.MLA_MAX_TABLE_ROWS + 1), dict(lens_from=None),
    dict(lens_to=None), dict(mean=None), dict(mean=P + 2), dict(device_flags=P + 2),
])
def test_blocks_mean_refuses(change):
    assert B.mla_blocks_mean(**{**MEAN, **change}) == B.MLA_EINVAL


SCORE = dict(batch=2, heads=16, q_latent=P, ql_token_stride=0, ql_head_stride=0, q_pe=P,
             qp_token_stride=0, qp_head_stride=0, q_scale_inv=None, mean=P, num_pages=16,
             page_size=64, block_table=P, bt_stride=8, table_rows=2, token_row=None, lens=P,
             scores=P, scores_stride=8, device_flags=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(batch=B.MLA_MAX_BATCH + 1), dict(heads=0),
    dict(heads=B.MLA_MAX_ROW_HEADS + 1), dict(q_latent=None), dict(q_latent=P + 8),
    dict(ql_head_stride=504), dict(ql_head_stride=516), dict(ql_token_stride=500),
    dict(q_pe=None), dict(qp_head_stride=60), dict(q_scale_inv=P, ql_head_stride=520), dict(mean=None),
    dict(num_pages=0), dict(page_size=0), dict(block_table=None), dict(bt_stride=0),
    dict(table_rows=0), dict(table_rows=1), dict(lens=None), dict(scores=None),
    dict(scores_stride=7), dict(q_scale_inv=P + 1),
])
def test_blocks_score_refuses(change):
    assert B.mla_blocks_score(**{**SCORE, **change}) == B.MLA_EINVAL


SELECT = dict(batch=2, scores=P, scores_stride=8, max_blocks=8, lens=P, page_size=64, keep_first=0,
              keep_last=1, k=4, sel=P, sel_stride=4, sel_count=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(batch=B.MLA_MAX_BATCH + 1), dict(scores=None), dict(scores=P + 2),
    dict(scores_stride=7), dict(max_blocks=0), dict(lens=None), dict(page_size=0),
    dict(keep_first=-1), dict(keep_last=-1), dict(k=0), dict(sel=None), dict(sel_stride=3),
    dict(sel_count=None),
])
def test_blocks_select_refuses(change):
    assert B.mla_blocks_select(**{**SELECT, **change}) == B.MLA_EINVAL


def test_attention_refuses_without_a_handle():
    h = ctypes.c_void_p()
    lib = B.load()
    for batch, heads in ((0, 16), (B.MLA_MAX_BATCH + 1, 16), (4, 0), (4, B.MLA_MAX_ROW_HEADS + 1)):
        assert lib.mla_attn_create(ctypes.byref(h), batch, heads) == B.MLA_EINVAL
    assert lib.mla_attn_create(None, 4, 16) == B.MLA_EINVAL
    assert h.value is None
    assert B.mla_attn_decode(None, 1, P, 0, 0, P, 0, 0, None, P, 4, 64, 0, P, P, 4, 1, None, P, None,
                             0, None, 0.1, P, 0, 0, None, None) == B.MLA_EINVAL
    with pytest.raises(B.MlaError):
        B.mla_attn_get_error(None)
    B.mla_attn_destroy(None)  # no-op


def test_runner_refuses_what_would_be_misread():
    """Types, inner strides and sizes are checked before a pointer is passed on."""
    i32 = torch.int32
    scores, lens = torch.zeros(2, 8), torch.ones(2, dtype=i32)
    sel, cnt = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in (dict(scores=scores.double()), dict(scores=torch.zeros(8, 2).T), dict(lens=lens.long()),
                dict(sel=sel.long()), dict(lens=lens[:1]), dict(cnt=cnt[:1])):
        a = dict(scores=scores, lens=lens, sel=sel, cnt=cnt) | bad
        with pytest.raises(B.MlaError):
            R.blocks_select(a["scores"], a["lens"], 64, 0, 0, a["sel"], a["cnt"], stream=0)
    cache, table = torch.zeros(4, 64, 576, dtype=torch.uint8), torch.zeros(2, 8, dtype=i32)
    mean, k_scale = torch.zeros(4, 576, dtype=torch.bfloat16), torch.ones(1)
    for bad in (dict(cache=cache[:, :, :575]), dict(layout=1), dict(mean=mean[:3]),
                dict(table=table.long()), dict(table=table[:1]), dict(layout=3)):
        a = dict(cache=cache, layout=0, k_scale=k_scale, table=table, mean=mean) | bad
        with pytest.raises(B.MlaError):
            R.blocks_mean(a["cache"], a["layout"], a["k_scale"], a["table"], lens, lens, a["mean"], stream=0)


def test_runner_refuses_tensors_off_the_device():
    """What would pass every other check, but lies in host memory, is refused before a launch."""
    i32 = torch.int32
    scores, lens, sel = torch.zeros(2, 8), torch.ones(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    cache, table = torch.zeros(4, 64, 576, dtype=torch.uint8), torch.zeros(2, 8, dtype=i32)
    mean, k_scale = torch.zeros(4, 576, dtype=torch.bfloat16), torch.ones(1)
    ql, qp = torch.zeros(2, 16, 512, dtype=torch.bfloat16), torch.zeros(2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: R.blocks_select(scores, lens, 64, 0, 0, sel, lens.clone(), stream=0),
                 lambda: R.blocks_mean(cache, 0, k_scale, table, lens, lens, mean, stream=0),
                 lambda: R.blocks_score(ql, qp, mean, 64, table, lens, scores, stream=0)):
        with pytest.raises(B.MlaError, match="device"):
            call()
    for bad in (lambda: R.blocks_select(None, lens, 64, 0, 0, sel, lens.clone(), stream=0),
                lambda: R.blocks_select(scores, [1, 1], 64, 0, 0, sel, lens.clone(), stream=0),
                lambda: R.blocks_select(scores, lens, "64", 0, 0, sel, lens.clone(), stream=0),
                lambda: R.blocks_select(scores, lens, 1 << 40, 0, 0, sel, lens.clone(), stream=0),
                lambda: R.blocks_score(ql[0], qp, mean, 64, table, lens, scores, stream=0),
                lambda: R.blocks_score(ql, qp.float(), mean, 64, table, lens, scores, stream=0)):
        with pytest.raises(B.MlaError):
            bad()
    with pytest.raises(B.MlaError, match="mean"):  # rows of another width
        R.blocks_score(ql, qp, mean.reshape(-1, 64), 64, table, lens, scores, stream=0)


def test_decode_takes_the_page_scaled_layout_only_with_scales():
    # a null handle is refused before the layout is looked at; the noalloc entry checks its layout itself
    args = [16, P, P, P, P, 1e-6, 1, P, 0, P, 0, P, 0, P, P, 4, 64, 3, None, P, P, None, None, None]
    assert B.mla_query_decode_noalloc(*args) == B.MLA_EINVAL
    args[17] = 4
    args[18] = P
    assert B.mla_query_decode_noalloc(*args) == B.MLA_EINVAL
