"""Host checks of the cache-side calls for torch tensors that have the right
sizes and types, but would be read or written elsewhere than they lie (CPU only:
every call here is refused before a launch, by the text that is matched)."""

import os

import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

BF16, I32 = torch.bfloat16, torch.int32
HERE = "tensors that are not on the current device"  # the last check: all else was taken


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mla_query_projection_gb300 import build

        build.build()
    return B.load()


def attend(tokens=3, heads=4, width=8, **change):
    """What the attention call says to these tensors in host memory; its handle is never followed."""
    a = dict(handle=4096, heads=heads, q_latent=torch.zeros(tokens, heads, 512, dtype=BF16),
             q_pe=torch.zeros(tokens, heads, 64, dtype=BF16), cache=torch.zeros(9, 16, 576, dtype=torch.uint8),
             layout=0, table=torch.zeros(tokens, width, dtype=I32), lens=torch.ones(tokens, dtype=I32), scale=0.1,
             k_scale=torch.ones(1), inv=None, token_row=None, sel=None, sel_count=None,
             out=torch.zeros(tokens, heads, 512, dtype=BF16), lse=None, stream=0)
    return R._native().attn_decode(*(a | change).values())


def score(tokens=3, heads=4, width=8, **change):
    a = dict(q_latent=torch.zeros(tokens, heads, 512, dtype=BF16), q_pe=torch.zeros(tokens, heads, 64, dtype=BF16),
             mean=torch.zeros(9, 576, dtype=BF16), page=16, table=torch.zeros(tokens, width, dtype=I32),
             lens=torch.ones(tokens, dtype=I32), scores=torch.zeros(tokens, width), inv=None, token_row=None, flags=None,
             stream=0)
    return R._native().blocks_score(*(a | change).values())


@pytest.mark.parametrize("call", [attend, score])
def test_broadcast_queries_are_refused(call):
    """An expanded tensor holds one token's or one head's rows: not what a row stride of 0 means to the library."""
    assert call() == HERE
    for name, width in (("q_latent", 512), ("q_pe", 64)):
        for shape in ((1, 4, width), (3, 1, width), (1, 1, width)):
            t = torch.zeros(shape, dtype=BF16).expand(3, 4, width)
            assert call(**{name: t}) == "query shape", (name, shape)
        # a single token or head is no broadcast, whatever its stride
        assert call(tokens=1, **{name: torch.zeros(1, 4, width, dtype=BF16).expand(1, 4, width)}) == HERE
        assert call(heads=1, **{name: torch.zeros(3, 1, width, dtype=BF16)}) == HERE
        odd = torch.zeros(8, 4, width, dtype=BF16).as_strided((1, 4, width), (7, width, 1))
        assert call(tokens=1, **{name: odd}) == HERE
    with pytest.raises(B.MlaError, match="query shape"):
        R.blocks_score(torch.zeros(1, 4, 512, dtype=BF16).expand(3, 4, 512), torch.zeros(3, 4, 64, dtype=BF16),
                       torch.zeros(9, 576, dtype=BF16), 16, torch.zeros(3, 8, dtype=I32), torch.ones(3, dtype=I32),
                       torch.zeros(3, 8), stream=0)


def test_broadcast_output_is_refused():
    assert attend(out=torch.zeros(1, 4, 512, dtype=BF16).expand(3, 4, 512)) == "out"
    assert attend(out=torch.zeros(3, 1, 512, dtype=BF16).expand(3, 4, 512)) == "out"
    assert attend(out=torch.zeros(4, 3, 512, dtype=BF16).transpose(0, 1)) == HERE  # head-major


def test_output_rows_that_overlap_are_refused():
    """Two heads or tokens written to the same place have no result."""
    room = torch.zeros(16 * 512, dtype=BF16)
    for strides in ((512, 512), (1024, 1024), (512, 1024), (3 * 512, 512), (512, 2 * 512)):
        assert attend(out=room.as_strided((3, 4, 512), (*strides, 1))) == "out", strides
    for strides in ((4 * 512, 512), (512, 3 * 512), (5 * 512, 512), (520, 3 * 520)):  # rows side by side, gaps
        assert attend(out=room.as_strided((3, 4, 512), (*strides, 1))) == HERE, strides


def test_columns_of_wider_tables():
    """The C calls take the columns apart from the stride: at least one, no more than the stride."""
    p = 4096
    mean = dict(kv_cache=p, num_pages=16, page_size=64, layout=0, k_scale=p, block_table=p, bt_stride=8, bt_cols=4,
                rows=2, lens_from=p, lens_to=p, mean=p, device_flags=None, stream=None)
    for bad in (dict(bt_cols=0), dict(bt_cols=9), dict(bt_cols=-1), dict(bt_stride=0, bt_cols=0), dict(mean=None)):
        assert B.mla_blocks_mean_cols(**(mean | bad)) == B.MLA_EINVAL
    assert B.mla_attn_decode_cols(None, 1, p, 0, 0, p, 0, 0, None, p, 4, 64, 0, p, p, 4, 2, 1, None, p, None, 0, 0, None,
                                  0.1, p, 0, 0, None, None) == B.MLA_EINVAL


def test_attention_without_an_output_refuses_what_is_no_query():
    attn = R.PagedAttention.__new__(R.PagedAttention)
    attn.handle, attn.heads = None, 4
    for q in (None, 3, torch.zeros(3, 4, 512, dtype=BF16)):
        with pytest.raises(B.MlaError):
            attn.decode(q, torch.zeros(3, 4, 64, dtype=BF16), torch.zeros(9, 16, 576, dtype=torch.uint8), 0,
                        torch.zeros(3, 8, dtype=I32), torch.ones(3, dtype=I32), 0.1, k_scale=torch.ones(1))


def test_decode_step_has_a_scale_for_every_page(monkeypatch):
    """With a scale a page, a step whose scales are fewer than its pages would have the kernel read behind them."""
    asked = []
    monkeypatch.setattr(B, "mla_query_decode", lambda *a: asked.append(a) or B.MLA_OK)
    step = R.DecodeStep.__new__(R.DecodeStep)
    step.handle = step.qkv_a = None
    step.batch, step.strides, step.layout = 1, (0, 0, 0), B.MLA_KV_FP8_E4M3_PAGE
    step.q_a = step.kv_c = step.k_pe = step.slots = step.cache = step.q_latent = step.q_pe = step.q_c = None
    step.num_pages, step.page_size = 8, 64
    for few in (torch.ones(1), torch.ones(7)):
        step.k_scale = few
        assert step.decode(stream=0) == B.MLA_EINVAL and not asked
    step.k_scale = torch.ones(16)[::2]  # eight, but not side by side
    assert step.decode(stream=0) == B.MLA_EINVAL and not asked
    step.k_scale = torch.ones(8)
    assert step.decode(stream=0) == B.MLA_OK and len(asked) == 1
    step.layout, step.k_scale = B.MLA_KV_FP8_E4M3, torch.ones(1)
    assert step.decode(stream=0) == B.MLA_OK and len(asked) == 2
