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


@pytest.mark.parametrize("layout,down", [(0, 0), (1, 0), (2, 0), (3, 0), (1, 8), (3, 8)])
def test_attention_keeps_the_sum_of_many_small_weights(layout, down):
    """One key beside 65,535 alike ones whose weights are 2^-11 to 2^-26 of its own (a range over the heads),
    in contexts that a worker reads whole; or weights 2^down times as large on rows of scales that much smaller.

    With w = 32 p a small weight as the kernel holds it (p of the large one), FP16 is off by 2^-11 w or
    2^-25, and the second term by a step of at most 2^-2 w, 2^-13 and at least 2^-16, once in 128 rows:
    they have the thresholds of that many parts of a step.  The large weight keeps 2^-7, the output 2^-8."""
    rng = np.random.default_rng(230 + layout)
    n, heads, tokens, page = 65536, 64, 152, 64
    pages = n // page
    row = np.zeros((n, C.ROW_BYTES[layout]), dtype=np.uint8)
    # latent values: one row for all, another for the sink; column 0 is zero
    code = lambda: (rng.integers(0, 2, 512) << 7 | rng.integers(4, 9, 512) << 3 | rng.integers(0, 8, 512)).astype(np.uint8)
    k_scale = np.full(pages if layout == 3 else 1, 0.125, dtype=np.float32)
    ratio = 2.0 ** -down
    for at, v in ((slice(None), 0.0), (5, 32.0)):
        if layout == 2:
            row[at, :256] = rng.integers(0, 256, 256)
            row[at, 0] &= 0xF0
            row[at, 256:288] = 7 << 3
            row[at, 288] = int(torch.tensor([v]).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            row[at, :512] = code()
            row[at, 0] = 0
            if layout == 1:
                row[at, 512:528] = np.full(4, 0.125 * (1.0 if v else ratio), dtype=np.float32).view(np.uint8)
                row[at, 528:530] = torch.tensor([v]).to(torch.bfloat16).view(torch.uint8).numpy()
            else:
                row[at, 512] = int(torch.tensor([v / 0.125]).to(torch.float8_e4m3fn).view(torch.uint8))
    cache = row.reshape(pages, page, -1)
    table = rng.permutation(pages).astype(np.int32)[None]
    if layout == 3:  # the sink's page keeps its scale
        k_scale[table[0, 1:]] *= np.float32(ratio)
    stored = np.empty_like(cache)
    stored[table[0]] = cache
    # logits: rope column 0 alone, 32 against 0; head h's small weights are 2^-bits[h]
    bits = np.linspace(11.0, 26.0, heads) - down
    ql, qp = torch.zeros(1, heads, 512, dtype=torch.bfloat16), torch.zeros(1, heads, 64, dtype=torch.bfloat16)
    ql[:, :, 0] = 1.0
    qp[0, :, 0] = torch.from_numpy(bits * np.log(2.0) / (SCALE * 32.0)).to(torch.bfloat16)
    q64 = torch.cat([ql, qp], 2).double().numpy()[0]
    keys = C.rows64(row[[100, 5]], layout, [0.125 * (ratio if layout == 3 else 1.0), 0.125])
    x = (q64 @ keys.T) * SCALE
    p = np.exp(x[:, 0] - x[:, 1])[:, None]
    total = 1.0 + (n - 1) * p
    count = n - 1.0  # of the small rows, in values of the ordinary one (those of the sink's page are larger)
    if layout == 3:
        count += (page - 1) * (1.0 / ratio - 1.0)
    want = (count * p * keys[0, :512] + keys[1, :512]) / total
    mass = (count * p * np.abs(keys[0, :512]) + np.abs(keys[1, :512])) / total
    attn = R.PagedAttention(tokens, heads)
    out, _ = attn.decode(ql.cuda().repeat(tokens, 1, 1), qp.cuda().repeat(tokens, 1, 1), dev(stored), layout, dev(table),
                         torch.full((tokens,), n, dtype=torch.int32, device="cuda"), SCALE, k_scale=dev(k_scale),
                         token_row=torch.zeros(tokens, dtype=torch.int32, device="cuda"))
    assert attn.error_flags() == 0
    attn.close()
    w = 32.0 * p * ratio
    each = 2.0 ** -11 * w + 2.0 ** -25
    if layout != 2:
        each = each + np.maximum(np.minimum(2.0 ** -2 * w, 2.0 ** -13), 2.0 ** -16) / 128
    each = n * each
    if down and layout == 3:  # the sink's page, each of its rows for itself
        each = each + page * (2.0 ** -13 + 2.0 ** -7 * w / ratio)
    slack = (2.0 ** -14.8 + 2.0 ** -17.8) * np.abs(x).max(1)[:, None] + (n / 256 + 16) * 2.0 ** -24
    bound = (each / 32.0 * np.abs(keys[0, :512]) / ratio + 2.0 ** -7 * np.abs(keys[1, :512])) / total \
        + 2 * slack * mass + 2.0 ** -8 * np.abs(want)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err.max(), (err / bound).max(), bits[np.argmax((err / bound).max((0, 2)))])


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("column", [0, 131, 511, 512, 575])
def test_attention_of_a_query_that_is_not_finite(layout, value, column):
    """It makes its head's results NaN, whatever the sign of the keys in its column, and no other's."""
    rng = np.random.default_rng(240 + column)
    heads, page = 33, 16
    cache, k_scale = C.make_cache(rng, 8, page, layout)
    where = [(p, o) for p in range(8) for o in range(page)]
    k = keys64(cache, k_scale, layout, where)[:, column]
    order = [int(np.argmax(k)), int(np.argmin(k))]  # a row of either sign in that column
    assert k[order[0]] > 0 > k[order[1]]
    # one request for each sign, of that row alone; one with all rows
    first = cache.reshape(128, -1)[order].copy()
    cache[6, 0], cache[7, 0] = first
    if layout == 3:
        k_scale[6], k_scale[7] = k_scale[[where[order[0]][0], where[order[1]][0]]]
    table = i32([[6, 0], [7, 0], [0, 1]])
    lens = i32([1, 1, 2 * page])
    ql, qp, _, _ = queries(rng, 3, heads)
    for t in range(3):
        if column < 512:
            ql[t, 17, column] = value
        else:
            qp[t, 17, column - 512] = value
    lse = torch.zeros(3, heads, device="cuda")
    attn = R.PagedAttention(3, heads)
    out, _ = attn.decode(ql, qp, dev(cache), layout, table, lens, SCALE, k_scale=dev(k_scale), lse=lse)
    assert attn.error_flags() == 0
    attn.close()
    others = [h for h in range(heads) if h != 17]
    for t in range(3):
        assert out[t, 17].isnan().all() and lse[t, 17].isnan(), t
        assert out[t, others].isfinite().all() and lse[t, others].isfinite().all(), t


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("latent", [0.0, 2.0 ** -40, 2.0 ** -12])
def test_attention_of_queries_whose_rope_part_is_far_larger(layout, latent):
    """Latent queries of zero, or far below the rope part: no product leaves FP32's range."""
    rng = np.random.default_rng(250)
    heads, page, n = 20, 16, 300
    pages = -(-n // page)
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    if layout == 1:
        pe = torch.from_numpy(rng.standard_normal((pages, page, 64), dtype=np.float32) * 3000.0).to(torch.bfloat16)
        cache[:, :, 528:] = pe.view(torch.uint8).numpy().reshape(pages, page, 128)
    table = C.make_table(rng, [n], page, pages)
    ql, qp, _, _ = queries(rng, 1, heads)
    ql, qp = (ql.float() * latent).to(torch.bfloat16), (qp.float() * 3000.0).to(torch.bfloat16)
    q64 = torch.cat([ql, qp], 2).double().cpu().numpy()
    where = C.positions(n, page, table.shape[1], pages, table[0])
    keys = keys64(cache, k_scale, layout, where)
    scale = float(np.float32(1.0 / np.abs(q64[0] @ keys.T).mean()))
    lse = torch.empty(1, heads, device="cuda")
    attn = R.PagedAttention(1, heads)
    out, _ = attn.decode(ql, qp, dev(cache), layout, dev(table), i32([n]), scale, k_scale=dev(k_scale), lse=lse)
    attn.close()
    check_attention(out[0], lse[0], q64[0], keys, scale, (layout, latent))


@pytest.mark.parametrize("stride", [1 << 33, 1 << 57, 1 << 62])
def test_a_single_row_may_have_any_stride(stride):
    """One request's table row: its stride leads nowhere, and stride * page_size does not fit 64 bits."""
    rng = np.random.default_rng(260)
    page, pages, heads, n = 64, 8, 16, 300
    cache, k_scale = C.make_cache(rng, pages, page, 0)
    table = C.make_table(rng, [n], page, pages)
    ql, qp, _, q64 = queries(rng, 1, heads)
    out = torch.zeros(1, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, heads, device="cuda")
    mean = torch.full((pages, 576), 9.0, dtype=torch.bfloat16, device="cuda")
    d = [dev(cache), dev(k_scale), dev(table), i32([n]), i32([0])]
    attn = R.PagedAttention(1, heads)
    stream = torch.cuda.current_stream()
    sel, count = i32([[4, 0]]), i32([2])
    where = C.positions(n, page, table.shape[1], pages, table[0])
    for s, sel_stride, c, w in ((None, 0, None, where),
                                (sel, stride, count, C.positions(n, page, table.shape[1], pages, table[0], [4, 0]))):
        rc = B.mla_attn_decode(attn.handle, 1, ql, 0, 0, qp, 0, 0, None, d[0], pages, page, 0, d[1], d[2], stride, 1, None,
                               d[3], s, sel_stride, c, SCALE, out, 0, 0, lse, stream)
        assert rc == B.MLA_OK and attn.error_flags() == 0
        check_attention(out[0], lse[0], q64[0], keys64(cache, k_scale, 0, w), SCALE, stride)
    rc = B.mla_blocks_mean(d[0], pages, page, 0, d[1], d[2], stride, 1, d[4], d[3], mean, None, stream)
    assert rc == B.MLA_OK
    torch.cuda.synchronize()
    got = mean.double().cpu().numpy()
    for j in range(-(-n // page)):
        k = keys64(cache, k_scale, 0, [(table[0, j], o) for o in range(min(page, n - j * page))])
        want, slack = k.mean(0), (page + 2) * 2.0 ** -24 * np.abs(k).mean(0)
        assert (np.abs(got[table[0, j]] - want) <= slack + 2.0 ** -8 * np.abs(want)).all()
    attn.close()


def test_attention_over_selected_blocks_flags_lengths_beyond_the_row():
    """As over the whole context: what the row holds is used, and the length flagged."""
    rng = np.random.default_rng(270)
    page, pages, heads, width = 16, 20, 16, 4
    cache, k_scale = C.make_cache(rng, pages, page, 0)
    table = rng.permutation(pages)[:3 * width].reshape(3, width).astype(np.int32)
    ql, qp, _, q64 = queries(rng, 3, heads)
    sel = [[3, 0], [1], []]
    lse = torch.zeros(3, heads, device="cuda")
    attn = R.PagedAttention(3, heads)
    for lens, flags in (([64, 20, 64], 0), ([65, 20, 64], B.MLA_DEVERR_BAD_SLOT), ([64, 20, 1000], B.MLA_DEVERR_BAD_SLOT)):
        out, _ = attn.decode(ql, qp, dev(cache), 0, dev(table), i32(lens), SCALE, k_scale=dev(k_scale), lse=lse,
                             sel=i32([[3, 0], [1, -1], [-1, -1]]), sel_count=i32([2, 1, 0]))
        assert attn.error_flags() == flags, lens
        for t, n in enumerate(lens):
            where = C.positions(n, page, width, pages, table[t], sel[t])
            check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, 0, where), SCALE, (t, n))
    attn.close()


def test_tables_step_given_back_more_pages_than_32_bits_count():
    """Requests that end with more pages in all than 2^32 (the same ones many times over): what the stack can
    hold, in row order, and no entry twice."""
    rows, page, pages, held = 4096, 1, 10000, (1 << 20) + 257  # those before the last one: 2^32 + 3839
    table = torch.arange(rows, dtype=torch.int32, device="cuda")[:, None].expand(rows, held).contiguous()
    lens = torch.full((rows,), held, dtype=torch.int32, device="cuda")
    new = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    stack = torch.full((pages,), -7, dtype=torch.int32, device="cuda")
    stack[:5] = torch.arange(9000, 9005)
    count, flags = i32([5]), i32([0])
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    token = [torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2)]
    cu = torch.full((rows + 1,), 9, dtype=torch.int32, device="cuda")
    R.tables_step(new, lens, table, stack, count, page, lens, count, slots, *token, cu, flags)
    assert int(count.item()) == pages and (lens == 0).all() and (cu == 0).all()
    assert stack[:5].tolist() == [9000, 9001, 9002, 9003, 9004]
    assert (stack[5:] == 0).all()  # the first request's, of which there are enough
    assert int(flags.item()) == B.MLA_DEVERR_REFUSED
    assert (slots == -1).all() and (token[0] == -1).all() and (token[1] == 0).all()
    del table
    torch.cuda.empty_cache()
