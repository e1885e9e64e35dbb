"""The cache-side operators on the GPU against their plain 64-bit forms
(tests/cache_ref.py), at the sizes and masks where they can go wrong.

Tolerances, derived before the first run.  Roundings are off by at most half a
step, relative to the value: BF16 2^-8, FP32 2^-24.
 * lse: with X = scale * sum_c |q_c k_c| (its largest over the keys), the FP32
   sum of 576 products is off by at most 576 * 2^-24 * X < 2^-14.8 X if every
   rounding fell the same way; queries split into two E4M3 terms keep each
   element to 2^-17.8 of the row's largest (test_attention's `q_split`), and
   the base-2 exponentials, the sum over n keys and the logarithm add at most
   (n / 256 + 16) * 2^-24 in relative terms to the sum.
 * out: a weight is rounded to BF16 (2^-8) or, where the kernel keeps it as the
   sum of an E4M3 and an E5M2 term, to 2^-4 * 2^-3 = 2^-7; so the output is off
   by at most (2^-7 + 2 * lse's bound) * sum_i p_i |c_i|, and its own rounding
   to BF16 adds 2^-8 |out|.
 * block means and scores: FP32 sums of at most 576 (page size) terms, and the
   mean's rounding to BF16.
Whole numbers are equal.
"""

import math

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

from . import cache_ref as C

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def cuda_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()
    torch.cuda.set_device(0)
    yield


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return t.to("cuda", dtype) if dtype is not None else t.to("cuda")


def queries(rng, tokens, heads, kind="bf16"):
    """(q_latent, q_pe, q_scale_inv or None) on the GPU and their FP64 rows [tokens, heads, 576]."""
    ql = torch.from_numpy(rng.standard_normal((tokens, heads, 512), dtype=np.float32) * 0.44)
    qp = torch.from_numpy(rng.standard_normal((tokens, heads, 64), dtype=np.float32) * 0.78)
    if kind == "bf16":
        ql, qp = ql.to(torch.bfloat16), qp.to(torch.bfloat16)
        return ql.cuda(), qp.cuda(), None, torch.cat([ql, qp], 2).double().numpy()
    inv = 32.0
    codes = [(x * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (ql, qp)]
    q64 = np.concatenate([C.E4M3[c.numpy()] for c in codes], 2) / inv
    return codes[0].cuda(), codes[1].cuda(), torch.tensor([inv], device="cuda"), q64


def keys64(cache, k_scale, layout, where):
    """FP64 keys of (page, offset) pairs."""
    if not where:
        return np.zeros((0, 576))
    p, o = np.array(where).T
    sc = k_scale[p] if layout == 3 else np.repeat(k_scale[:1], len(p))
    return C.rows64(cache[p, o], layout, sc)


def check_attention(out, lse, q64, keys, scale, label):
    o, want_lse, mass, mag = C.attend64(q64, keys, scale)
    n = len(keys)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    if n == 0:
        assert (out == 0).all() and np.isneginf(lse).all(), label
        return
    qmax, kl1 = np.abs(q64).max(1), np.abs(keys).sum(1).max()
    q_split = 2.0 ** -17.8 * qmax * kl1 * scale
    slack = 2.0 ** -14.8 * mag + q_split + (n / 256 + 16) * 2.0 ** -24
    assert np.isfinite(lse).all(), label
    assert (np.abs(lse - want_lse) <= slack + 2.0 ** -23 * np.abs(want_lse)).all(), (
        label, np.abs(lse - want_lse).max(), slack.min())
    bound = (2.0 ** -7 + 2 * slack)[:, None] * mass + 2.0 ** -8 * np.abs(o) + 1e-30
    err = np.abs(out - o)
    assert (err <= bound).all(), (label, err.max(), (err / bound).max())


def run_attention(rng, lens, heads, layout, page, kind="bf16", sel=None, token_row=None, rows=None,
                  spare=3, width=None, garbage=True, attn=None):
    """Attention of tokens with these lengths; `rows`: the requests' lengths where tokens share them."""
    req = list(lens) if rows is None else list(rows)
    pages = sum(-(-max(int(n), 0) // page) for n in req) + spare
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    table = C.make_table(rng, [max(0, n) for n in req], page, pages, width)
    if garbage:  # NaN codes wherever no request's position lies
        live = np.zeros((pages, page), dtype=bool)
        for r, n in enumerate(req):
            for p, o in C.positions(n, page, table.shape[1], pages, table[r]):
                live[p, o] = True
        cache[~live] = 0x7F if layout != 1 else 0xFF
    tokens = len(lens)
    ql, qp, inv, q64 = queries(rng, tokens, heads, kind)
    own = attn is None
    attn = attn or R.PagedAttention(tokens, heads)
    lse = torch.full((tokens, heads), float("nan"), device="cuda")
    out = torch.full((tokens, heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = cnt = None
    if sel is not None:
        k = max(1, max(len(x) for x in sel))
        arr = np.full((tokens, k), -1, dtype=np.int32)
        for t, x in enumerate(sel):
            arr[t, :len(x)] = x
        s, cnt = dev(arr), dev(np.array([len(x) for x in sel], dtype=np.int32))
    attn.decode(ql, qp, dev(cache), layout, dev(table), dev(np.array(lens, dtype=np.int32)), SCALE,
                k_scale=dev(k_scale), q_scale_inv=inv,
                token_row=None if token_row is None else dev(np.array(token_row, dtype=np.int32)),
                sel=s, sel_count=cnt, out=out, lse=lse)
    torch.cuda.synchronize()
    flags = attn.error_flags()
    for t, n in enumerate(lens):
        r = t if token_row is None else token_row[t]
        where = C.positions(n, page, table.shape[1], pages, table[r] if 0 <= r < len(table) else [-1] * table.shape[1],
                            None if sel is None else sel[t])
        check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, layout, where), SCALE,
                        (t, n, heads, layout, page, kind))
    if own:
        attn.close()
    return flags


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("heads", [1, 16, 17, 32, 64, 100, 128])
def test_attention_heads_and_layouts(layout, heads):
    rng = np.random.default_rng(100 * layout + heads)
    assert run_attention(rng, [1, 130, 0, 700], heads, layout, 64) == 0


@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 100, 128, 256])
@pytest.mark.parametrize("layout,kind", [(0, "bf16"), (1, "e4m3"), (2, "bf16"), (3, "e4m3")])
def test_attention_page_sizes(page, layout, kind):
    rng = np.random.default_rng(7000 + 10 * page + layout)
    assert run_attention(rng, [63, 64, 65, 127, 128, 129, 385], 64, layout, page, kind) == 0


@pytest.mark.parametrize("heads,kind", [(16, "bf16"), (64, "bf16"), (64, "e4m3"), (128, "e4m3")])
@pytest.mark.parametrize("layout", [0, 1])
def test_attention_one_long_context(layout, heads, kind):
    """Every worker holds a part of one token's context."""
    rng = np.random.default_rng(31 + heads)
    assert run_attention(rng, [30011], heads, layout, 64, kind) == 0


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
def test_attention_ragged_batch(layout):
    rng = np.random.default_rng(55 + layout)
    lens = [int(x) for x in rng.integers(0, 900, 61)] + [0, 2500, 1]
    assert run_attention(rng, lens, 128, layout, 64) == 0


@pytest.mark.parametrize("heads", [200, 1024])
def test_attention_gathered_heads(heads):
    """More heads than one rank has: several head groups."""
    rng = np.random.default_rng(heads)
    assert run_attention(rng, [300, 0, 77], heads, 0, 64) == 0


@pytest.mark.parametrize("layout,kind", [(0, "bf16"), (1, "bf16"), (2, "e4m3"), (3, "e4m3")])
@pytest.mark.parametrize("page", [16, 64, 100])
def test_attention_selected_blocks(layout, kind, page):
    """Selections in any order, one named twice, blocks outside the row and beyond the length,
    and none at all."""
    rng = np.random.default_rng(900 + page + layout)
    lens = [page * 9 + 5, page * 4, 3, page * 30 + 1, page * 2]
    sel = [[9, 0, 4, 4], [3, 7, 1, -1], [0], list(range(30, -1, -2)), []]
    assert run_attention(rng, lens, 64, layout, page, kind, sel=sel, width=33) == 0


def test_attention_tokens_share_requests():
    """Several tokens of a request, each with its own causal length; a padded token."""
    rng = np.random.default_rng(12)
    rows = [300, 65]
    lens = [297, 298, 299, 300, 64, 65, 0]
    assert run_attention(rng, lens, 64, 0, 64, token_row=[0, 0, 0, 0, 1, 1, -1], rows=rows) == 0


def test_attention_flags_what_the_table_cannot_hold():
    """Absent pages, lengths beyond the row and rows outside the table are left out, with a flag."""
    rng = np.random.default_rng(13)
    page, pages = 16, 12
    cache, k_scale = C.make_cache(rng, pages, page, 0)
    table = np.array([[3, -1, 5, 99], [1, 2, 4, 6]], dtype=np.int32)
    lens, token_row = [60, 200, 30], [0, 1, 2]
    ql, qp, inv, q64 = queries(rng, 3, 64)
    attn = R.PagedAttention(3, 64)
    lse = torch.empty(3, 64, device="cuda")
    out, _ = attn.decode(ql, qp, dev(cache), 0, dev(table), dev(np.array(lens, dtype=np.int32)), SCALE,
                         k_scale=dev(k_scale), token_row=dev(np.array(token_row, dtype=np.int32)), lse=lse)
    assert attn.error_flags() == B.MLA_DEVERR_BAD_SLOT
    assert attn.error_flags() == 0  # read and cleared
    for t, r in enumerate(token_row):
        where = C.positions(lens[t], page, 4, pages, table[r]) if r < 2 else []
        check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, 0, where), SCALE, t)
    attn.close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_gathered_rows_and_strided_output(kind):
    """Query rows [B][q_heads][576] at a head offset, outputs head-major."""
    rng = np.random.default_rng(14)
    heads, q_heads, off = 24, 64, 32
    cache, k_scale = C.make_cache(rng, 8, 64, 0)
    table, lens = np.array([[0, 1, 2], [3, 4, 5]], dtype=np.int32), [130, 40]
    ql, qp, inv, q64 = queries(rng, 2, heads, kind)
    rows = torch.zeros(2, q_heads, 576, dtype=ql.dtype, device="cuda")
    rows[:, off:off + heads, :512], rows[:, off:off + heads, 512:] = ql, qp
    out = torch.empty(heads, 2, 512, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.empty(2, heads, device="cuda")
    attn = R.PagedAttention(2, heads)
    attn.decode(rows[:, off:off + heads, :512], rows[:, off:off + heads, 512:], dev(cache), 0, dev(table),
                dev(np.array(lens, dtype=np.int32)), SCALE, k_scale=dev(k_scale), q_scale_inv=inv, out=out, lse=lse)
    for t in range(2):
        where = C.positions(lens[t], 64, 3, 8, table[t])
        check_attention(out[t], lse[t], q64[t], keys64(cache, k_scale, 0, where), SCALE, t)
    attn.close()


@pytest.mark.parametrize("layout", [0, 1, 2])
def test_attention_offsets_beyond_32_bits(layout):
    """Pages at byte offsets beyond 2^32 of the cache."""
    rng = np.random.default_rng(15)
    page, row = 64, C.ROW_BYTES[layout]
    pages = (1 << 32) // (page * row) + 40
    small, k_scale = C.make_cache(rng, 6, page, layout)
    cache = torch.empty(pages, page, row, dtype=torch.uint8, device="cuda")
    at = [pages - 1, 2, pages - 7, pages - 20, 0, pages - 3]
    for i, p in enumerate(at):
        cache[p] = dev(small[i])
    table = np.array([at], dtype=np.int32)
    ql, qp, inv, q64 = queries(rng, 1, 64)
    attn = R.PagedAttention(1, 64)
    lse = torch.empty(1, 64, device="cuda")
    out, _ = attn.decode(ql, qp, cache, layout, dev(table), dev(np.array([350], dtype=np.int32)), SCALE,
                         k_scale=dev(k_scale), lse=lse)
    where = [(i, o) for i in range(6) for o in range(page) if i * page + o < 350]
    check_attention(out[0], lse[0], q64[0], keys64(small, k_scale, layout, where), SCALE, layout)
    attn.close()


@pytest.mark.parametrize("layout,page", [(0, 64), (1, 64), (2, 64), (3, 64), (0, 7), (1, 12), (2, 1), (3, 100)])
def test_attention_growing_maximum_and_a_sink(layout, page):
    """The largest logit comes late, and one key (a sink) outweighs thousands of others: the running
    maximum has to grow, and small weights have to keep their sum."""
    rng = np.random.default_rng(16 + layout)
    n, heads = 6000, 64
    pages = -(-n // page)
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    table = C.make_table(rng, [n], page, pages)
    q64 = np.zeros((1, heads, 576))
    ql = torch.from_numpy(rng.standard_normal((1, heads, 512), dtype=np.float32) * 0.2).to(torch.bfloat16)
    qp = torch.zeros(1, heads, 64, dtype=torch.bfloat16)
    qp[0, :, 0] = 2.0
    where = C.positions(n, page, table.shape[1], pages, table[0])
    # rope value 0 of a key: grows with the position, the last key far above all
    for i, (p, o) in enumerate(where):
        v = 8.0 * i / n + (64.0 if i == n - 5 else 0.0)
        if layout == 2:
            cache[p, o, 288] = int(torch.tensor([v]).to(torch.float8_e4m3fn).view(torch.uint8))
        elif layout == 1:
            cache[p, o, 528:530] = torch.tensor([v]).to(torch.bfloat16).view(torch.uint8).numpy()
        else:
            sc = float(k_scale[p] if layout == 3 else k_scale[0])
            code = torch.tensor([min(448.0, v / sc)]).to(torch.float8_e4m3fn).view(torch.uint8)
            cache[p, o, 512] = int(code)
    q64[0] = torch.cat([ql, qp], 2).double().numpy()[0]
    attn = R.PagedAttention(1, heads)
    lse = torch.empty(1, heads, device="cuda")
    out, _ = attn.decode(ql.cuda(), qp.cuda(), dev(cache), layout, dev(table), dev(np.array([n], dtype=np.int32)),
                         SCALE, k_scale=dev(k_scale), lse=lse)
    check_attention(out[0], lse[0], q64[0], keys64(cache, k_scale, layout, where), SCALE, layout)
    attn.close()


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,width", [(64, 4000), (64, 400), (7, 20000)])
def test_attention_tables_far_wider_than_the_requests(layout, kind, page, width):
    """What a table could hold decides on the heads a CTA takes; the lengths stay short."""
    rng = np.random.default_rng(50 + layout)
    assert run_attention(rng, [300, 0, 77, 1, 513], 100, layout, page, kind, width=width) == 0


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("page", [16, 100])
def test_attention_workers_with_several_tokens(layout, page):
    """Many tiles a worker (ten groups of heads leave each 15 workers), and tokens that end inside their shares."""
    rng = np.random.default_rng(60 + layout)
    lens = [1, 0, 900, 128, 129, 2000, 5, 640, 0, 1300, 127, 1025, 3, 3000, 2100]
    assert run_attention(rng, lens, 640, layout, page) == 0


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("page", [1, 64])
def test_attention_full_batch(layout, page):
    """As many tokens as a call takes, most of them short, empty ones among them."""
    rng = np.random.default_rng(40 + layout)
    lens = [int(n) for n in rng.integers(0, 40, B.MLA_MAX_BATCH)]
    lens[0], lens[17], lens[100], lens[255] = 1, 1500, 0, 129
    assert run_attention(rng, lens, 16, layout, page) == 0


@pytest.mark.parametrize("ratio", [1.0, 1.3, 0.0])
def test_attention_scales_that_differ(ratio):
    """fp8_ds_mla scales a row apart by up to 2^12, by no power of two, and zero in some rows.

    (Scaled weights go through FP16 twice, 2^-11 each: 2^-7 + 2^-10 of a weight at
    most, and 2^-24 of a plane's largest row for what falls below FP16's steps.)"""
    rng = np.random.default_rng(45)
    n, heads, page = 700, 64, 64
    cache, k_scale = C.make_cache(rng, 12, page, 1)
    table = C.make_table(rng, [n], page, 12)
    sc = np.exp2(-rng.integers(0, 13, (12, page, 4))).astype(np.float32) * np.float32(0.02 * max(ratio, 1.0))
    if ratio == 0.0:
        sc[rng.random(sc.shape) < 0.2] = 0.0
    cache[:, :, 512:528] = sc.view(np.uint8).reshape(12, page, 16)
    ql, qp, inv, q64 = queries(rng, 1, heads)
    where = C.positions(n, page, table.shape[1], 12, table[0])
    keys = keys64(cache, k_scale, 1, where)
    attn = R.PagedAttention(1, heads)
    lse = torch.empty(1, heads, device="cuda")
    out, _ = attn.decode(ql, qp, dev(cache), 1, dev(table), dev(np.array([n], dtype=np.int32)), SCALE, lse=lse)
    assert attn.error_flags() == 0
    attn.close()
    o, want_lse, mass, mag = C.attend64(q64[0], keys, SCALE)
    slack = 2.0 ** -14.8 * mag + 2.0 ** -17.8 * np.abs(q64[0]).max(1) * np.abs(keys).sum(1).max() * SCALE \
        + (n / 256 + 16) * 2.0 ** -24
    assert (np.abs(lse[0].double().cpu().numpy() - want_lse) <= slack + 2.0 ** -23 * np.abs(want_lse)).all()
    err = np.abs(out[0].double().cpu().numpy() - o)
    floor = n * 2.0 ** -24 * 448 * float(sc.max())
    assert (err <= (2.0 ** -7 + 2.0 ** -10 + 2 * slack)[:, None] * mass + 2.0 ** -8 * np.abs(o) + floor).all(), err.max()


@pytest.mark.parametrize("order", ["up", "down", "zeros"])
def test_attention_page_scales_that_differ(order):
    """Page scales apart by 2^12, the larger ones later or earlier, or zero on most pages, the first ones too.

    (Weights are kept over the largest scale of a worker's first tile, to steps of
    2^-16 at a largest weight of 2^5 or more: n * 2^-22 of the largest value.)"""
    rng = np.random.default_rng(48)
    n, heads, page = 1500, 64, 16
    pages = -(-n // page) + 2
    cache, k_scale = C.make_cache(rng, pages, page, 3)
    table = C.make_table(rng, [n], page, pages)
    blocks = -(-n // page)
    sc = 0.03 * np.exp2(12.0 * np.arange(blocks) / blocks - 12.0)
    if order == "down":
        sc = sc[::-1]
    if order == "zeros":
        sc = np.where((np.arange(blocks) < 40) | (rng.random(blocks) < 0.5), 0.0, 0.03)
    k_scale[table[0, :blocks]] = sc.astype(np.float32)
    ql, qp, inv, q64 = queries(rng, 1, heads)
    where = C.positions(n, page, table.shape[1], pages, table[0])
    keys = keys64(cache, k_scale, 3, where)
    attn = R.PagedAttention(1, heads)
    lse = torch.empty(1, heads, device="cuda")
    out, _ = attn.decode(ql, qp, dev(cache), 3, dev(table), dev(np.array([n], dtype=np.int32)), SCALE,
                         k_scale=dev(k_scale), lse=lse)
    assert attn.error_flags() == 0
    attn.close()
    o, want_lse, mass, mag = C.attend64(q64[0], keys, SCALE)
    slack = 2.0 ** -14.8 * mag + 2.0 ** -17.8 * np.abs(q64[0]).max(1) * np.abs(keys).sum(1).max() * SCALE \
        + (n / 256 + 16) * 2.0 ** -24
    assert (np.abs(lse[0].double().cpu().numpy() - want_lse) <= slack + 2.0 ** -23 * np.abs(want_lse)).all()
    err = np.abs(out[0].double().cpu().numpy() - o)
    floor = n * 2.0 ** -22 * 448 * float(k_scale.max())
    assert (err <= (2.0 ** -7 + 2 * slack)[:, None] * mass + 2.0 ** -8 * np.abs(o) + floor).all(), err.max()


def test_attention_of_a_nan_row():
    """A NaN in a row that counts reaches the heads' results, in that token only."""
    rng = np.random.default_rng(46)
    for layout in (0, 1, 2, 3):
        cache, k_scale = C.make_cache(rng, 4, 64, layout)
        table = np.array([[0, 1], [2, 3]], dtype=np.int32)
        cache[1, 5] = 0x7F if layout != 1 else 0xFF
        ql, qp, inv, q64 = queries(rng, 2, 16)
        attn = R.PagedAttention(2, 16)
        out, _ = attn.decode(ql, qp, dev(cache), layout, dev(table), dev(np.array([100, 100], dtype=np.int32)), SCALE,
                             k_scale=dev(k_scale))
        assert out[0].isnan().all(), layout
        assert not out[1].isnan().any(), layout
        attn.close()


def test_attention_two_handles_at_once():
    """Calls of two handles run side by side on two streams; graphs of one handle follow one another."""
    rng = np.random.default_rng(47)
    cache, k_scale = C.make_cache(rng, 200, 64, 3)
    table = dev(C.make_table(rng, [6000, 6100], 64, 200))
    cache, k_scale = dev(cache), dev(k_scale)
    lens = [dev(np.array(x, dtype=np.int32)) for x in ([6000, 6100], [3001, 17])]
    ql, qp, inv, q64 = queries(rng, 2, 128)
    attn = [R.PagedAttention(2, 128) for _ in range(2)]
    want = []
    for a, n in zip(attn, lens):
        want.append(a.decode(ql, qp, cache, 3, table, n, SCALE, k_scale=k_scale)[0])
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(want[0]) for _ in range(2)]
    for _ in range(20):
        for a, n, s, o in zip(attn, lens, streams, outs):
            with torch.cuda.stream(s):
                a.decode(ql, qp, cache, 3, table, n, SCALE, k_scale=k_scale, out=o)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)
        o.zero_()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, n, o in zip(graphs, lens, outs):  # both on the first handle's workspace
        with torch.cuda.graph(g):
            attn[0].decode(ql, qp, cache, 3, table, n, SCALE, k_scale=k_scale, out=o)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)
    for a in attn:
        a.close()


def test_attention_repeats_and_streams():
    """The same bits from call to call, from another stream and from a replayed graph with new lengths."""
    rng = np.random.default_rng(17)
    cache, k_scale = C.make_cache(rng, 64, 64, 0)
    table = C.make_table(rng, [1900, 1800], 64, 64)
    ql, qp, inv, q64 = queries(rng, 2, 64)
    args = [dev(cache), 0, dev(table)]
    lens = dev(np.array([1900, 1000], dtype=np.int32))
    kw = dict(k_scale=dev(k_scale), lse=torch.empty(2, 64, device="cuda"))
    attn = R.PagedAttention(2, 64)
    first = attn.decode(ql, qp, *args, lens, SCALE, **kw)[0].clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    with torch.cuda.stream(other):
        attn.decode(ql, qp, *args, lens, SCALE, out=out, **kw)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.decode(ql, qp, *args, lens, SCALE, out=out, **kw)
    out.zero_()
    graph.replay()
    assert torch.equal(first, out)
    lens.copy_(torch.tensor([5, 1800], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for t, n in enumerate([5, 1800]):
        where = C.positions(n, 64, table.shape[1], 64, table[t])
        check_attention(out[t], kw["lse"][t], q64[t], keys64(cache, k_scale, 0, where), SCALE, t)
    attn.close()


def test_attention_right_behind_what_writes_its_lengths():
    """Lengths that the call before wrote, a step after another in one graph: every step sees its own."""
    rng = np.random.default_rng(49)
    rows, page, pages = 3, 16, 300
    cache, k_scale = C.make_cache(rng, pages, page, 0)
    ql, qp, inv, q64 = queries(rng, rows, 16)
    cache_d, scale_d = dev(cache), dev(k_scale)
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    table = torch.full((rows, 90), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pages, dtype=torch.int32, device="cuda"), dev(np.array([pages], dtype=np.int32))
    news = [[900, 5, 0], [1, 1, 300], [1, 500, 1], [200, 1, 1]]
    steps = [dict(new=dev(np.array(n, dtype=np.int32)), slots=torch.zeros(1500, dtype=torch.int64, device="cuda"),
                  row=torch.zeros(1500, dtype=torch.int32, device="cuda"),
                  ln=torch.zeros(1500, dtype=torch.int32, device="cuda"),
                  out=torch.zeros(rows, 16, 512, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.zeros(rows, 16, device="cuda")) for n in news]
    cu = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
    attn = R.PagedAttention(rows, 16)

    def go():
        for s in steps:
            R.tables_step(s["new"], lens, table, free, count, page, lens, count, s["slots"], s["row"], s["ln"], cu)
            attn.decode(ql, qp, cache_d, 0, table, lens, SCALE, k_scale=scale_d, out=s["out"], lse=s["lse"])

    go()  # (and once more below, from a graph)
    lens.zero_()
    table.fill_(-1)
    free.copy_(torch.arange(pages, dtype=torch.int32))
    count.fill_(pages)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    graph.replay()
    torch.cuda.synchronize()
    assert attn.error_flags() == 0
    final, held = table.cpu().numpy(), np.zeros(rows, dtype=int)
    for s, n in zip(steps, news):
        held += n
        for r in range(rows):
            where = C.positions(int(held[r]), page, 90, pages, final[r])
            check_attention(s["out"][r], s["lse"][r], q64[r], keys64(cache, k_scale, 0, where), SCALE, (n, r))
    attn.close()


def test_attention_refuses_more_tokens_than_its_workspace():
    attn = R.PagedAttention(1, 16)
    ql, qp, _, _ = queries(np.random.default_rng(1), 2, 16)
    cache, table = torch.zeros(2, 64, 576, dtype=torch.uint8).cuda(), torch.zeros(2, 1, dtype=torch.int32).cuda()
    lens = torch.ones(2, dtype=torch.int32).cuda()
    host = torch.ones(2, dtype=torch.int32)  # lengths in host memory
    with pytest.raises(B.MlaError):
        attn.decode(ql[:1], qp[:1], cache, 0, table, host, SCALE, k_scale=torch.ones(1).cuda())
    for kw in (dict(), dict(sel=table)):  # too many tokens; a selection without its counts
        with pytest.raises(B.MlaError):
            attn.decode(ql, qp, cache, 0, table, lens, SCALE, k_scale=torch.ones(1).cuda(), **kw)
    with pytest.raises(B.MlaError):  # one token, but a scale that is not finite
        attn.decode(ql[:1], qp[:1], cache, 0, table, lens[:1], float("nan"), k_scale=torch.ones(1).cuda())
    with pytest.raises(B.MlaError):  # no stream
        attn.decode(ql[:1], qp[:1], cache, 0, table, lens[:1], SCALE, k_scale=torch.ones(1).cuda(), stream="1")
    attn.close()
    with pytest.raises(B.MlaError):
        attn.decode(ql[:1], qp[:1], cache, 0, table, lens[:1], SCALE, k_scale=torch.ones(1).cuda())


# ------------------------------------------------------------------- tables


def step(new, lens, table, stack, count, page, max_tokens, alias=False):
    d = dict(new=dev(np.array(new, dtype=np.int32)), lens=dev(np.array(lens, dtype=np.int32)), table=dev(table),
             stack=dev(stack), count=dev(np.array([count], dtype=np.int32)),
             slots=torch.full((max_tokens,), 77, dtype=torch.int64, device="cuda"),
             row=torch.full((max_tokens,), 77, dtype=torch.int32, device="cuda"),
             ln=torch.full((max_tokens,), 77, dtype=torch.int32, device="cuda"),
             cu=torch.full((len(lens) + 1,), 77, dtype=torch.int32, device="cuda"),
             flags=torch.zeros(1, dtype=torch.int32, device="cuda"))
    d["lens_out"] = d["lens"] if alias else torch.full_like(d["lens"], 77)
    d["count_out"] = d["count"] if alias else torch.full_like(d["count"], 77)
    R.tables_step(d["new"], d["lens"], d["table"], d["stack"], d["count"], page, d["lens_out"], d["count_out"],
                  d["slots"], d["row"], d["ln"], d["cu"], d["flags"])
    return d


def check_step(d, ref):
    got = dict(lens=d["lens_out"], table=d["table"], stack=d["stack"], slots=d["slots"], token_row=d["row"],
               token_len=d["ln"], cu=d["cu"])
    for k, v in got.items():
        np.testing.assert_array_equal(v.cpu().numpy(), np.asarray(ref[k]), err_msg=k)
    assert int(d["count_out"].item()) == ref["count"]
    assert bool(d["flags"].item() & B.MLA_DEVERR_REFUSED) == ref["refused"]


def state(rng, lens, page, pages, width):
    table = C.make_table(rng, lens, page, pages, width)
    used = set(table[table >= 0].tolist())
    free = [p for p in rng.permutation(pages) if p not in used]
    stack = np.full(pages, -1, dtype=np.int32)
    stack[:len(free)] = free
    return table, stack, len(free)


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("rows,page,width,longest,tokens", [
    (1, 64, 4, 1, 1), (5, 1, 9, 3, 64), (64, 64, 12, 1, 64), (64, 16, 40, 200, 4000), (300, 7, 30, 20, 9000),
    (513, 64, 8, 60, 2048), (1000, 64, 5, 1, 1000), (4096, 16, 6, 9, 4096 * 9), (40, 16, 40, 200, 3003),
    (7, 48, 30, 300, 257),
])
def test_tables_step(rows, page, width, longest, tokens, alias):
    rng = np.random.default_rng(rows + page)
    lens = rng.integers(0, max(2, page * width // 2), rows)
    new = rng.integers(0, longest + 1, rows)
    new[rng.random(rows) < 0.1] = -1
    pages = int(sum(-(-n // page) for n in lens)) + rows * (longest // page + 2)
    table, stack, count = state(rng, lens, page, pages, width)
    d = step(new, lens, table, stack, count, page, tokens, alias)
    check_step(d, C.tables_ref(new, lens, table, stack, count, page, tokens))


@pytest.mark.parametrize("tokens", [63, 3001])
def test_tables_step_into_unaligned_arrays(tokens):
    """Token arrays that begin one entry into their allocation; what lies around them stays."""
    rng = np.random.default_rng(70)
    rows, page, width = 20, 16, 30
    lens = rng.integers(0, 100, rows).astype(np.int32)
    new = rng.integers(0, 4 if tokens < 100 else 140, rows).astype(np.int32)
    pages = 600
    table = C.make_table(rng, [int(n) for n in lens], page, pages, width)
    held = set(table[r, j] for r in range(rows) for j in range(-(-int(lens[r]) // page)))
    stack = np.full(pages, -7, dtype=np.int32)
    free = [p for p in range(pages) if p not in held]
    stack[:len(free)] = free
    want = C.tables_ref(new, lens, table, stack, len(free), page, tokens)
    d = step(new, lens, table, stack, len(free), page, tokens)
    check_step(d, want)
    wide = dict(slots=torch.full((tokens + 9,), 55, dtype=torch.int64, device="cuda"),
                row=torch.full((tokens + 9,), 55, dtype=torch.int32, device="cuda"),
                ln=torch.full((tokens + 9,), 55, dtype=torch.int32, device="cuda"))
    cut = {k: v[1:1 + tokens] for k, v in wide.items()}
    again = torch.zeros_like(d["lens_out"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    R.tables_step(dev(new), dev(lens), dev(table), dev(stack), dev(np.array([len(free)], dtype=np.int32)), page,
                  again[0], again[1], cut["slots"], cut["row"], cut["ln"],
                  torch.zeros(rows + 1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for k, v in cut.items():
        assert torch.equal(v, d[k]), k
        assert (wide[k][:1] == 55).all() and (wide[k][1 + tokens:] == 55).all(), k


@pytest.mark.parametrize("what", ["pages", "tokens", "row", "length"])
@pytest.mark.parametrize("rows", [6, 700])
def test_tables_step_refuses_requests(what, rows):
    """Too few pages, too little room, a full table row, an unsound length: as documented, the rest served."""
    rng = np.random.default_rng(rows)
    page, width = 16, 6
    lens = rng.integers(0, 60, rows)
    new = rng.integers(1, 30, rows)
    new[rows // 2] = -1
    pages = int(sum(-(-n // page) for n in lens)) + (0 if what == "pages" else 4 * rows)
    tokens = int(new.clip(0).sum()) + 5
    if what == "tokens":
        tokens = int(new[: rows // 3].clip(0).sum()) + 3
    if what == "row":
        lens[rows // 4], new[rows // 4] = 80, 30
    table, stack, count = state(rng, lens, page, pages, width)
    if what == "length":
        lens[1], lens[rows - 1] = -3, page * width + 1
        new[rows - 1] = -1
    d = step(new, lens, table, stack, count, page, tokens)
    ref = C.tables_ref(new, lens, table, stack, count, page, tokens)
    assert ref["refused"]
    check_step(d, ref)


def test_tables_steps_in_a_graph():
    """Replayed in place, the state advances step by step."""
    rng = np.random.default_rng(3)
    rows, page, width, pages = 9, 4, 30, 200
    lens = rng.integers(0, 20, rows)
    new = np.array([1, 2, 0, 1, -1, 5, 1, 1, 3])
    table, stack, count = state(rng, lens, page, pages, width)
    d = step(np.zeros(rows), lens, table, stack, count, page, 16, alias=True)
    d["new"].copy_(dev(new.astype(np.int32)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.tables_step(d["new"], d["lens"], d["table"], d["stack"], d["count"], page, d["lens"], d["count"],
                      d["slots"], d["row"], d["ln"], d["cu"], d["flags"])
    for _ in range(5):
        graph.replay()
        ref = C.tables_ref(new, lens, table, stack, count, page, 16)
        check_step(d, ref)
        lens, table, stack, count = ref["lens"], ref["table"], ref["stack"], ref["count"]


# ------------------------------------------------------------- block choice


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("page", [1, 7, 64, 100])
def test_blocks_mean(layout, page):
    rng = np.random.default_rng(page + layout)
    to = [0, 1, page, page + 1, 5 * page - 1, 3 * page]
    frm = [0, 0, 0, page, 2 * page + 1, 3 * page]
    pages = sum(-(-n // page) for n in to) + 2
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    table = C.make_table(rng, to, page, pages, 6)
    mean = torch.full((pages, 576), 9.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.blocks_mean(dev(cache), layout, dev(k_scale), dev(table), dev(np.array(frm, dtype=np.int32)),
                  dev(np.array(to, dtype=np.int32)), mean, flags)
    got = mean.double().cpu().numpy()
    want, slack = np.full((pages, 576), 9.0), np.zeros((pages, 576))
    for r, (a, b) in enumerate(zip(frm, to)):
        for j in range(a // page, -(-b // page)):
            p = table[r, j]
            k = keys64(cache, k_scale, layout, [(p, o) for o in range(min(page, b - j * page))])
            want[p] = k.mean(0)
            # page + 2 FP32 roundings of a sum, at most half a step of the magnitudes each
            slack[p] = (page + 2) * 2.0 ** -24 * np.abs(k).mean(0)
    assert (np.abs(got - want) <= slack + 2.0 ** -8 * np.abs(want) + 1e-30).all()
    assert int(flags.item()) == 0


@pytest.mark.parametrize("heads", [1, 16, 33, 128, 200])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_blocks_score(heads, kind):
    rng = np.random.default_rng(heads)
    page, pages, width = 16, 90, 41
    mean = torch.from_numpy(rng.standard_normal((pages, 576), dtype=np.float32)).to(torch.bfloat16)
    lens = [41 * 16, 1, 0, 16, 17 * 16 + 3]
    table = np.array([rng.permutation(pages)[:width] for _ in lens], dtype=np.int32)
    table[4, 3] = -1
    ql, qp, inv, q64 = queries(rng, 5, heads, kind)
    scores = torch.full((5, 50), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.blocks_score(ql, qp, mean.cuda(), page, dev(table), dev(np.array(lens, dtype=np.int32)), scores,
                   q_scale_inv=inv, flags=flags)
    got = scores.double().cpu().numpy()
    m64 = mean.double().numpy()
    for t, n in enumerate(lens):
        for j in range(width):
            if j * page >= n or table[t, j] < 0:
                assert np.isneginf(got[t, j])
                continue
            prod = q64[t] @ m64[table[t, j]]
            bound = 577 * 2.0 ** -24 * (np.abs(q64[t]) @ np.abs(m64[table[t, j]])).max()
            assert abs(got[t, j] - prod.max()) <= bound
    assert (got[:, width:] == 7.0).all()
    assert int(flags.item()) == B.MLA_DEVERR_BAD_SLOT


@pytest.mark.parametrize("n,k", [(1, 1), (1, 4), (5, 5), (31, 8), (512, 100), (513, 512), (1500, 1), (9000, 700)])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_blocks_select(n, k, kind):
    rng = np.random.default_rng(n + k)
    s = rng.standard_normal((3, n)).astype(np.float32)
    if kind == "ties":
        s = np.round(s)
    if kind == "special":
        s[rng.random(s.shape) < 0.3] = np.nan
        s[rng.random(s.shape) < 0.2] = -np.inf
        s[rng.random(s.shape) < 0.1] = np.inf
        s[rng.random(s.shape) < 0.2] = -0.0
        s[rng.random(s.shape) < 0.2] = 0.0
    page, first, last = 4, n % 3, (n + 1) % 4
    lens = np.array([n * page, max(0, n * page // 2 - 1), 0], dtype=np.int32)
    sel = torch.full((3, k), 55, dtype=torch.int32, device="cuda")
    cnt = torch.full((3,), 55, dtype=torch.int32, device="cuda")
    R.blocks_select(dev(s), dev(lens), page, first, last, sel, cnt)
    for t in range(3):
        want = C.select_ref(s[t], -(-int(lens[t]) // page), first, last, k)
        assert int(cnt[t]) == len(want)
        assert sel[t].tolist() == want + [-1] * (k - len(want))


# ------------------------------------------------------------------ together


def test_page_scaled_insert_equals_the_tensor_scaled_one():
    """A row of the page-scaled layout has the bytes that the per-tensor layout gives with the page's scale."""
    from mla_query_projection_gb300 import synthetic as S
    from mla_query_projection_gb300.runner import DecodeStep

    for batch, heads in ((1, 16), (5, 16), (12, 64), (40, 64)):
        inp = S.make_inputs(batch=batch, heads=heads, layout=S.LAYOUT_E4M3, pages=8, seed=40 + batch)
        st = DecodeStep(inp)
        cache0 = st.cache.clone()
        scales = torch.linspace(0.01, 0.2, 8, device="cuda")
        want = cache0.clone()
        for p in range(8):
            st.cache.copy_(cache0)
            st.k_scale.copy_(scales[p])
            assert st.decode() == B.MLA_OK
            torch.cuda.synchronize()
            want[p] = st.cache[p]
        st.cache.copy_(cache0)
        st.k_scale, st.layout = scales, B.MLA_KV_FP8_E4M3_PAGE
        assert st.decode() == B.MLA_OK
        torch.cuda.synchronize()
        assert st.error_flags() == 0
        assert torch.equal(st.cache, want)
        st.close()


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
def test_steps_of_a_serving_loop(layout):
    """Tables, decode, means, scores, selection and attention, step after step: the slots the tables give
    are the rows the attention reads, dense and over the selected blocks."""
    from mla_query_projection_gb300 import synthetic as S
    from mla_query_projection_gb300.runner import DecodeStep

    rng = np.random.default_rng(layout)
    rows, page, pages, width, heads, k = 6, 8, 64, 10, 16, 3
    S_LAYOUT = 0 if layout == 3 else layout
    tokens = 8
    inp = S.make_inputs(batch=tokens, heads=heads, layout=S_LAYOUT, pages=pages, page_size=page, seed=90 + layout)
    st = DecodeStep(inp)
    st.layout = layout
    st.k_scale = torch.rand(pages, device="cuda") * 0.1 + 0.02 if layout == 3 else st.k_scale
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    stack = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
    trow, tlen = (torch.empty(tokens, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = torch.empty(rows + 1, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    mean = torch.zeros(pages, 576, dtype=torch.bfloat16, device="cuda")
    scores = torch.empty(tokens, width, device="cuda")
    sel, cnt = torch.empty(tokens, k, dtype=torch.int32, device="cuda"), torch.empty(tokens, dtype=torch.int32, device="cuda")
    attn = R.PagedAttention(tokens, heads)
    lse = torch.empty(tokens, heads, device="cuda")
    st.slots = slots
    for i in range(12):
        new = torch.tensor([1, 2, 0, 1, 1, 1] if i != 7 else [1, -1, 3, 1, -1, 1], dtype=torch.int32, device="cuda")
        before = lens.clone()
        R.tables_step(new, lens, table, stack, count, page, lens, count, slots, trow, tlen, cu, flags)
        st.q_a.normal_()
        st.kv_c.normal_()
        st.k_pe.normal_()
        assert st.decode() == B.MLA_OK
        before = torch.minimum(before, lens)
        R.blocks_mean(st.cache, layout, st.k_scale, table, before, lens, mean, flags)
        R.blocks_score(st.q_latent, st.q_pe, mean, page, table, tlen, scores, token_row=trow, flags=flags)
        R.blocks_select(scores, tlen, page, 1, 1, sel, cnt)
        dense, _ = attn.decode(st.q_latent, st.q_pe, st.cache, layout, table, tlen, SCALE, k_scale=st.k_scale,
                               token_row=trow, lse=lse)
        torch.cuda.synchronize()
        dense_lse = lse.clone()
        sparse, _ = attn.decode(st.q_latent, st.q_pe, st.cache, layout, table, tlen, SCALE, k_scale=st.k_scale,
                                token_row=trow, sel=sel, sel_count=cnt, lse=lse)
        torch.cuda.synchronize()
        assert st.error_flags() == 0 and attn.error_flags() == 0 and int(flags.item()) == 0
        cache, ks, tab = st.cache.cpu().numpy(), st.k_scale.cpu().numpy(), table.cpu().numpy()
        q64 = torch.cat([st.q_latent, st.q_pe], 2).double().cpu().numpy()
        total = int(cu[-1])
        for t in range(tokens):
            r, n = int(trow[t]), int(tlen[t])
            assert (r >= 0) == (t < total) and (int(slots[t]) >= 0) == (t < total)
            row = tab[r] if r >= 0 else [-1] * width
            if t < total:
                assert int(slots[t]) == row[(n - 1) // page] * page + (n - 1) % page
            where = C.positions(n, page, width, pages, row)
            check_attention(dense[t], dense_lse[t], q64[t], keys64(cache, ks, layout, where), SCALE, (i, t))
            blocks = sel[t, :int(cnt[t])].tolist()
            nb = -(-n // page)
            assert blocks == C.select_ref(scores[t].cpu().numpy(), nb, 1, 1, k)
            where = C.positions(n, page, width, pages, row, blocks)
            check_attention(sparse[t], lse[t], q64[t], keys64(cache, ks, layout, where), SCALE, (i, t, "sparse"))
            assert math.isfinite(float(lse[t, 0])) == (n > 0)
    attn.close()
    st.close()
