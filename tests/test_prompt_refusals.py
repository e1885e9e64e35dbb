"""Host checks of the prompt's entry points: what the documentation rules out is
refused before anything reaches the device (CPU only)."""

import ctypes
import math
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
INV = [10000.0 ** (-i / 32) for i in range(32)]


@pytest.fixture(scope="module")
def rope():
    h = B.mla_rope_create(INV)
    yield h
    B.mla_rope_destroy(h)


@pytest.mark.parametrize("change", [
    dict(inv_freq=INV[:31]), dict(inv_freq=[math.nan] + INV[1:]), dict(inv_freq=[math.inf] + INV[1:]),
    dict(inv_freq=[2e6] + INV[1:]), dict(axis=[0] * 31), dict(axis=[-1] + [0] * 31),
    dict(axis=[B.MLA_MAX_ROPE_AXES] + [0] * 31), dict(axis=[2 ** 40] + [0] * 31), dict(scale=math.nan),
    dict(scale=math.inf),
])
def test_rope_create_refuses(change):
    with pytest.raises(B.MlaError):
        B.mla_rope_create(**{**dict(inv_freq=INV, axis=None, interleaved=True, scale=1.0), **change})


def test_rope_create_without_arrays():
    h = ctypes.c_void_p()
    lib = B.load()
    assert lib.mla_rope_create(None, None, None, 1, 1.0) == B.MLA_EINVAL
    assert lib.mla_rope_create(ctypes.byref(h), None, None, 1, 1.0) == B.MLA_EINVAL
    assert h.value is None
    assert B.mla_rope_axes(None) == B.MLA_EINVAL
    B.mla_rope_destroy(None)  # no-op
    several = B.mla_rope_create(INV, [0, 4] + [2] * 30)
    assert B.mla_rope_axes(several) == 5
    B.mla_rope_destroy(several)


APPLY = dict(tokens=3, heads=4, x=P, x_token_stride=0, x_head_stride=0, positions=P, pos_stride=0, pos_offset=0, out=P,
             out_token_stride=0, out_head_stride=0, stream=None)


@pytest.mark.parametrize("change", [
    dict(handle=None), dict(tokens=-1), dict(heads=0), dict(heads=B.MLA_MAX_ROW_HEADS + 1), dict(x=None), dict(out=None),
    dict(positions=None), dict(x=P + 8), dict(out=P + 2), dict(positions=P + 2), dict(x_head_stride=60),
    dict(x_head_stride=68), dict(x_token_stride=-256), dict(out_token_stride=260), dict(out_head_stride=8),
    dict(pos_stride=2), dict(pos_offset=2 ** 31), dict(pos_offset=-2 ** 31 - 1),
])
def test_rope_apply_refuses(rope, change):
    assert B.mla_rope_apply(**{**dict(handle=rope), **APPLY, **change}) == B.MLA_EINVAL


@pytest.mark.parametrize("change", [dict(x_head_stride=2 ** 62), dict(x_token_stride=2 ** 38), dict(out_head_stride=2 ** 61),
                                    dict(out_token_stride=2 ** 38)])
def test_rope_apply_refuses_strides_beyond_any_memory(rope, change):
    assert B.mla_rope_apply(**{**dict(handle=rope), **APPLY, "heads": 128, **change}) == B.MLA_EINVAL


def test_cache_write_refuses_tokens_beyond_any_memory():
    assert B.mla_cache_write(**{**WRITE, "tokens": 2 ** 63 - 1}) == B.MLA_EINVAL


def test_calls_of_nothing_do_nothing(rope):
    assert B.mla_rope_apply(**{**dict(handle=rope), **APPLY, "tokens": 0, "x": None, "out": None}) == B.MLA_OK
    assert B.mla_cache_write(**{**WRITE, "tokens": 0, "kv_c": None}) == B.MLA_OK
    assert B.mla_cache_read(**{**READ, "max_rows": 0, "rows": None}) == B.MLA_OK


WRITE = dict(tokens=3, kv_c=P, kv_c_stride=0, k_pe=P, k_pe_stride=0, gamma_kv=P, eps=1e-6, rope=None, positions=None,
             pos_stride=0, pos_offset=0, slot_mapping=P, kv_cache=P, num_pages=4, page_size=64, layout=0, k_scale=P,
             rows=P, rows_stride=0, device_flags=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(kv_c=None), dict(k_pe=None), dict(slot_mapping=None), dict(kv_cache=None), dict(k_scale=None),
    dict(layout=3, k_scale=None), dict(layout=4), dict(layout=-1), dict(num_pages=0), dict(page_size=0),
    dict(num_pages=2 ** 60), dict(eps=-1.0), dict(eps=math.nan), dict(kv_c_stride=504), dict(kv_c_stride=516),
    dict(k_pe_stride=56), dict(k_pe_stride=68), dict(rows_stride=568), dict(rows_stride=580), dict(kv_c=P + 8),
    dict(k_pe=P + 8), dict(gamma_kv=P + 8), dict(kv_cache=P + 8), dict(rows=P + 8), dict(slot_mapping=P + 4),
    dict(k_scale=P + 2), dict(device_flags=P + 2), dict(positions=P),
])
def test_cache_write_refuses(change):
    assert B.mla_cache_write(**{**WRITE, **change}) == B.MLA_EINVAL


@pytest.mark.parametrize("change", [dict(positions=None), dict(pos_stride=2), dict(pos_offset=2 ** 31), dict(positions=P + 2)])
def test_cache_write_refuses_rotations(rope, change):
    assert B.mla_cache_write(**{**WRITE, "rope": rope, "positions": P, **change}) == B.MLA_EINVAL


READ = dict(kv_cache=P, num_pages=4, page_size=64, layout=0, k_scale=P, block_table=P, bt_stride=4, bt_cols=4, requests=2,
            cu_rows=P, first=P, max_rows=10, rows=P, rows_stride=0, device_flags=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(kv_cache=None), dict(num_pages=0), dict(page_size=0), dict(num_pages=2 ** 60), dict(layout=4), dict(k_scale=None),
    dict(block_table=None), dict(bt_cols=0), dict(bt_cols=5), dict(requests=0), dict(requests=B.MLA_MAX_TABLE_ROWS + 1),
    dict(cu_rows=None), dict(max_rows=-1), dict(max_rows=2 ** 31), dict(rows=None), dict(rows_stride=568),
    dict(rows_stride=580), dict(kv_cache=P + 8), dict(rows=P + 8), dict(block_table=P + 2), dict(cu_rows=P + 2),
    dict(first=P + 1), dict(device_flags=P + 3), dict(k_scale=P + 1),
])
def test_cache_read_refuses(change):
    assert B.mla_cache_read(**{**READ, **change}) == B.MLA_EINVAL


def test_prompt_attention_refuses_without_a_handle():
    h = ctypes.c_void_p()
    lib = B.load()
    assert lib.mla_prompt_create(None, 16) == B.MLA_EINVAL
    for heads in (0, -1, B.MLA_MAX_ROW_HEADS + 1):
        assert lib.mla_prompt_create(ctypes.byref(h), heads) == B.MLA_EINVAL
    assert h.value is None
    assert B.mla_prompt_attn(None, 1, 4, 4, P, 0, 0, P, 0, 0, P, 0, 0, P, 0, P, 0, 0, P, P, 1, None, 0.1, 0.0, None, P, 0, 0,
                             None, None) == B.MLA_EINVAL
    with pytest.raises(B.MlaError):
        B.mla_prompt_get_error(None)
    B.mla_prompt_destroy(None)  # no-op


def test_runner_refuses_what_would_be_misread():
    """Types, shapes and strides are checked before a pointer is passed on; host tensors last."""
    bf, i32 = torch.bfloat16, torch.int32
    rot = R.Rotary(INV)
    x, pos, out = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(3, 4, 64, dtype=bf)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x[..., :63]), dict(pos=pos.long()), dict(pos=pos[:2]),
                dict(pos=torch.zeros(6, dtype=i32)[::2]), dict(out=out[:2]), dict(out=out.float()), dict(x=None),
                dict(out=torch.zeros(3, 1, 64, dtype=bf).expand(3, 4, 64)), dict(offset=2 ** 31), dict(offset="1"),
                dict(x=torch.zeros(1, 4, 64, dtype=bf).expand(3, 4, 64))):
        a = dict(x=x, pos=pos, out=out, offset=0) | bad
        with pytest.raises(B.MlaError):
            rot.apply(a["x"], a["pos"], out=a["out"], offset=a["offset"], stream=0)
    with pytest.raises(B.MlaError, match="device"):
        rot.apply(x, pos, out=out, stream=0)
    several = R.Rotary(INV, [0, 1] * 16)
    for bad in (pos, torch.zeros(1, 3, dtype=i32), torch.zeros(2, 2, dtype=i32)):
        with pytest.raises(B.MlaError, match="positions"):
            several.apply(x, bad, out=out, stream=0)

    kv, pe, slots = torch.zeros(3, 512, dtype=bf), torch.zeros(3, 64, dtype=bf), torch.zeros(3, dtype=torch.int64)
    cache, rows, scale = torch.zeros(2, 4, 576, dtype=torch.uint8), torch.zeros(3, 576, dtype=bf), torch.ones(1)
    good = dict(kv_c=kv, k_pe=pe, slot_mapping=slots, cache=cache, layout=0, k_scale=scale, rows=rows, stream=0)
    for bad in (dict(kv_c=kv[:2]), dict(kv_c=kv[:, :511]), dict(kv_c=kv.float()), dict(k_pe=pe[:2]), dict(k_pe=kv),
                dict(slot_mapping=slots.int()), dict(cache=cache[..., :575]), dict(layout=1), dict(layout=3),
                dict(k_scale=scale.double()), dict(rows=rows[:2]), dict(rows=kv), dict(gamma=kv[0, :511]),
                dict(rotary=rot), dict(positions=pos), dict(rotary=rot, positions=pos[:2]), dict(eps="x"),
                dict(flags=slots), dict(kv_c=torch.zeros(1, 512, dtype=bf).expand(3, 512))):
        with pytest.raises(B.MlaError):
            R.cache_write(**{**good, **bad})
    with pytest.raises(B.MlaError, match="device"):
        R.cache_write(**good)
    table, cu = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32)
    good = dict(cache=cache, layout=0, k_scale=scale, block_table=table, cu_rows=cu, rows=rows, stream=0)
    for bad in (dict(block_table=table[:1]), dict(block_table=table.long()), dict(cu_rows=cu[:1]), dict(cu_rows=cu.long()),
                dict(rows=rows[:, :575]), dict(rows=rows.float()), dict(first=cu[:1]), dict(first=cu.long()),
                dict(layout=2), dict(layout=3), dict(rows=torch.zeros(1, 576, dtype=bf).expand(3, 576))):
        with pytest.raises(B.MlaError):
            R.cache_read(**{**good, **bad})
    with pytest.raises(B.MlaError, match="device"):
        R.cache_read(**good)
    rot.close()
    with pytest.raises(B.MlaError, match="closed"):
        rot.apply(x, pos, out=out, stream=0)
    with pytest.raises(B.MlaError, match="closed"):
        R.cache_write(**{**dict(kv_c=kv, k_pe=pe, slot_mapping=slots, cache=cache, layout=0, k_scale=scale, stream=0),
                         "rotary": rot, "positions": pos})
