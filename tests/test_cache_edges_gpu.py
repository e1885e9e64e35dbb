"""The cache-side operators on the GPU in calls that lie at the edge of what the
documentation allows: views, streams, small weights, infinities.  Plain 64-bit
forms and tolerances as in test_cache_ops_gpu.py, others beside their tests."""

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

from . import cache_ref as C
from .test_cache_ops_gpu import SCALE, check_attention, dev, keys64, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()
    torch.cuda.set_device(0)
    yield


def i32(x):
    return dev(np.array(x, dtype=np.int32))


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("first", [0, 2, 8])
def test_attention_over_columns_of_a_wider_table(layout, first):
    """Only the view's columns count: lengths beyond them are flagged, and blocks behind them left out."""
    rng = np.random.default_rng(200 + layout)
    page, pages, heads, stride, width = 16, 40, 20, 12, 4
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    wide = np.array([rng.permutation(pages)[:stride] for _ in range(3)], dtype=np.int32)
    view = dev(wide)[:, first:first + width]
    assert first + width <= stride and view.stride(0) == stride
    ql, qp, _, q64 = queries(rng, 3, heads)
    attn = R.PagedAttention(3, heads)
    lse = torch.empty(3, heads, device="cuda")
    for lens, flags in (([64, 5, 33], 0), ([64, 150, 65], B.MLA_DEVERR_BAD_SLOT)):
        out, _ = attn.decode(ql, qp, dev(cache), layout, view, i32(lens), SCALE, k_scale=dev(k_scale), lse=lse)
        assert attn.error_flags() == flags
        for t, n in enumerate(lens):
            where = C.positions(n, page, width, pages, wide[t, first:first + width])
            check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, layout, where), SCALE, (t, n))
    # selections: blocks from the view's width on are outside the row; counts beyond the view's columns are cut
    chosen = np.array([[3, 4, 1, 0, 0], [0, 7, 2, 3, 1], [1, 1, 5, 2, 3]], dtype=np.int32)
    lens = [64, 60, 50]
    out, _ = attn.decode(ql, qp, dev(cache), layout, view, i32(lens), SCALE, k_scale=dev(k_scale), lse=lse,
                         sel=dev(chosen)[:, :3], sel_count=i32([3, 5, 2]))
    for t, n in enumerate(lens):
        where = C.positions(n, page, width, pages, wide[t, first:first + width], chosen[t, :[3, 3, 2][t]].tolist())
        check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, layout, where), SCALE, (t, n, "selected"))
    attn.close()


@pytest.mark.parametrize("layout", [0, 2])
def test_blocks_mean_over_columns_of_a_wider_table(layout):
    rng = np.random.default_rng(210 + layout)
    page, pages, stride, first, width = 16, 40, 12, 8, 4
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    wide = rng.permutation(pages)[:3 * stride].reshape(3, stride).astype(np.int32)
    mean = torch.full((pages, 576), 9.0, dtype=torch.bfloat16, device="cuda")
    to = [10, 64, 500]  # the last one longer than the view
    R.blocks_mean(dev(cache), layout, dev(k_scale), dev(wide)[:, first:first + width], i32([0, 0, 0]), i32(to), mean)
    got, want, slack = mean.double().cpu().numpy(), np.full((pages, 576), 9.0), np.zeros((pages, 576))
    for r, n in enumerate(to):
        for j in range(width):
            fill = min(page, n - j * page)
            if fill > 0:
                p = wide[r, first + j]
                k = keys64(cache, k_scale, layout, [(p, o) for o in range(fill)])
                want[p], slack[p] = k.mean(0), (page + 2) * 2.0 ** -24 * np.abs(k).mean(0)
    assert (np.abs(got - want) <= slack + 2.0 ** -8 * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("form", ["stream", "handle", "default"])
def test_attention_output_belongs_to_the_calls_stream(form):
    """An output that the call allocates is memory of the stream that it runs on: not a block that the
    current stream has given back, whose work there may not be done."""
    rng = np.random.default_rng(220)
    cache, k_scale = C.make_cache(rng, 8, 64, 0)
    table = C.make_table(rng, [400, 30], 64, 8)
    ql, qp, _, q64 = queries(rng, 2, 64)
    args = (ql, qp, dev(cache), 0, dev(table), i32([400, 30]), SCALE)
    lse, scale = torch.empty(2, 64, device="cuda"), dev(k_scale)
    attn = R.PagedAttention(2, 64)
    other, current = torch.cuda.Stream(), torch.cuda.Stream()
    given = {"stream": other, "handle": other.cuda_stream, "default": 0}[form]
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        free = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")  # given back to the current stream
        at = free.data_ptr()
        del free
        out, _ = attn.decode(*args, k_scale=scale, lse=lse, stream=given)
        assert out.data_ptr() != at
        again = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")
        assert again.data_ptr() == at
    torch.cuda.synchronize()
    assert attn.error_flags() == 0
    for t, n in enumerate((400, 30)):
        where = C.positions(n, 64, table.shape[1], 8, table[t])
        check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, 0, where), SCALE, (t, form))
    with torch.cuda.stream(current):  # without one, the current stream's
        assert attn.decode(*args, k_scale=scale, lse=lse)[0].data_ptr() not in (at, out.data_ptr())
    torch.cuda.synchronize()
    attn.close()
