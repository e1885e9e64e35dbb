"""The row operators of a prompt on the GPU (rotary positions, cache rows written
and read back) against their plain 64-bit forms.

Tolerances, derived before the first run.  Half a step of BF16 is 2^-8 of a value.
 * rotation: the angle's turns are kept to 2^-64 a position, then to 2^-32 of a
   turn and, as FP32 half turns, to 2^-25 of a half turn: 2^-23.3 radians; sine
   and cosine add 2 ulp (2^-22 at most), the scale, products and sums three
   roundings.  So a value is off by less than 2^-20 scale (|x0| + |x1|) before
   its own rounding to BF16 (2^-8 |y|).
 * normalised rows: FP32 arithmetic of 512 terms, 2^-14 at most, far less than the
   rounding to BF16; rows must equal the decode step's bytes, whose own parity the
   oracle checks, or the oracle's row functions.
 * rows read back: a code times its scale, rounded to FP32 and then to BF16:
   2^-8 + 2^-24 of the value.
"""

import math

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R
from mla_query_projection_gb300 import synthetic as S
from oracle import mla_oracle as O

from . import cache_ref as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()
    torch.cuda.set_device(0)
    yield


def inv_freq(theta=10000.0):
    return theta ** (-np.arange(0, 64, 2) / 64.0)


def turned64(x, pos, inv, axis, interleaved, scale=1.0, offset=0):
    """x [tokens, heads, 64] (FP64), pos [axes, tokens]: the turned rows, and scale (|x0| + |x1|)."""
    x, pos = np.asarray(x, dtype=np.float64), np.atleast_2d(np.asarray(pos, dtype=np.int64)) + offset
    y, mag = np.empty_like(x), np.empty_like(x)
    for p in range(32):
        # the angle in turns, from exact integer arithmetic: the frequency as a fraction of 2^80
        f = int(math.floor(inv[p] / (2 * math.pi) * 2 ** 80))
        turns = np.array([float(((int(v) * f) % 2 ** 80) / 2 ** 80) for v in pos[axis[p]]])
        a = 2 * math.pi * turns
        co, si = np.cos(a)[:, None], np.sin(a)[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + 32)
        y[..., i] = scale * (x[..., i] * co - x[..., j] * si)
        y[..., j] = scale * (x[..., j] * co + x[..., i] * si)
        mag[..., i] = mag[..., j] = abs(scale) * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return y, mag


def check_turned(got, x, pos, inv, axis, interleaved, scale=1.0, offset=0):
    # inv / (2 pi) is itself off by 2^-52 of it: a position's angle by 2^-52 |pos| inv
    want, mag = turned64(x, pos, inv, axis, interleaved, scale, offset)
    far = np.abs(np.asarray(pos, dtype=np.float64) + offset).max() * np.abs(inv).max()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + far * 2.0 ** -51) * mag + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * std).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 128), (3, 7), (64, 128), (65, 16), (1000, 1), (5, 1000), (2500, 9)])
def test_rope_shapes(tokens, heads, interleaved):
    rng = np.random.default_rng(tokens + heads)
    x, pos = bf16(rng, tokens, heads, 64), rng.integers(0, 70000, tokens).astype(np.int32)
    inv = inv_freq()
    rot = R.Rotary(inv, interleaved=interleaved)
    assert rot.axes == 1
    out = rot.apply(x, torch.from_numpy(pos).cuda())
    check_turned(out, x.double().cpu(), pos, inv, [0] * 32, interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_several_axes_scale_and_offset(interleaved):
    rng = np.random.default_rng(5)
    axis = rng.integers(0, 3, 32)
    axis[7] = 2
    pos = rng.integers(-3000, 3000, (3, 40)).astype(np.int32)
    inv, x = inv_freq(), bf16(rng, 40, 12, 64)
    rot = R.Rotary(inv, axis, interleaved, scale=0.75)
    assert rot.axes == 3
    wide = torch.full((4, 50), 9, dtype=torch.int32, device="cuda")  # a wider array's first columns
    wide[:3, :40] = torch.from_numpy(pos).cuda()
    out = rot.apply(x, wide[:, :40], offset=-17)
    check_turned(out, x.double().cpu(), pos, inv, axis, interleaved, 0.75, -17)


def test_rope_negative_frequencies_turn_as_negative_positions():
    """The same turns, so the same bytes, however small the frequency and far the position."""
    rng = np.random.default_rng(8)
    x, inv = bf16(rng, 2000, 16, 64), 10.0 ** rng.uniform(-8, 0, 32)
    pos = torch.from_numpy(rng.integers(-2 ** 31 + 1, 2 ** 31, 2000).astype(np.int32)).cuda()
    assert torch.equal(R.Rotary(-inv).apply(x, pos), R.Rotary(inv).apply(x, -pos))


def test_rope_far_positions_and_frequencies_from_none_to_many():
    rng = np.random.default_rng(6)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 24 + 1], dtype=np.int32)
    inv = np.concatenate([[0.0, 1.0, 2 * math.pi, 1e6, -0.5, 1e-9], inv_freq()[:26]])
    x = bf16(rng, len(pos), 3, 64)
    out = R.Rotary(inv).apply(x, torch.from_numpy(pos).cuda())
    # (pair by pair: the largest frequency would loosen every bound)
    for p in range(32):
        only = np.zeros(32)
        only[p] = inv[p]
        want, mag = turned64(x.double().cpu(), pos, only, [0] * 32, True)
        i = slice(2 * p, 2 * p + 2)
        far = np.abs(pos.astype(np.float64))[:, None, None] * abs(inv[p])
        tol = 2.0 ** -8 * np.abs(want[..., i]) + (2.0 ** -20 + far * 2.0 ** -51) * mag[..., i] + 1e-38
        assert (np.abs(out.double().cpu().numpy()[..., i] - want[..., i]) <= tol).all(), p


def test_rope_in_place_in_gathered_rows_and_back():
    """Gathered rows' rope part, turned in place; the other parts stay; minus the positions turns back."""
    rng = np.random.default_rng(7)
    rows = bf16(rng, 20, 24, 576)
    before = rows.clone()
    pos = torch.arange(1000, 1020, dtype=torch.int32, device="cuda")
    rot = R.Rotary(inv_freq())
    got = rot.apply(rows[..., 512:], pos, out=rows[..., 512:])
    assert got.data_ptr() == rows[..., 512:].data_ptr()
    assert torch.equal(rows[..., :512], before[..., :512])
    check_turned(rows[..., 512:], before[..., 512:].double().cpu(), pos.cpu().numpy(), inv_freq(), [0] * 32, True)
    back = rot.apply(rows[..., 512:], -pos)
    # a second rounding to BF16: twice half a step of the pair's length
    x = before[..., 512:].double()
    length = (x.unflatten(-1, (32, 2)).square().sum(-1).sqrt()).repeat_interleave(2, -1)
    assert ((back.double() - x).abs() <= 2 * 2.0 ** -8 * length * 2 ** 0.5).all()


def test_rope_of_fused_rows_and_no_tokens():
    rng = np.random.default_rng(8)
    row = bf16(rng, 33, 2112)
    k_pe = row[:, None, 2048:]
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    out = R.Rotary(inv_freq(), interleaved=False).apply(k_pe, pos)
    check_turned(out, k_pe.double().cpu(), np.arange(33), inv_freq(), [0] * 32, False)
    none = R.Rotary(inv_freq()).apply(row[:0, None, 2048:], pos[:0])
    assert none.shape == (0, 1, 64)


# ---------------------------------------------------------------- cache_write


def write_case(layout, tokens, pages=40, page=64, seed=0, fused=True):
    inp = S.make_inputs(batch=tokens, heads=1, layout=layout if layout < 3 else 0, pages=pages, seed=seed,
                        page_size=page, row_scale=True)
    if layout == 3:
        inp["layout"] = 3
        inp["k_scale"] = np.random.default_rng(seed).uniform(0.01, 0.2, pages).astype(np.float32)
    inp["slots"][::5] = -1
    return inp


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("tokens", [1, 9, 64, 256])
def test_cache_write_equals_the_decode_steps_bytes(layout, tokens):
    inp = write_case(layout, tokens, seed=tokens)
    step = R.DecodeStep(inp, fused_row=True)
    cache = step.cache.clone()
    assert step.decode() == B.MLA_OK
    rows = torch.full((tokens, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.cache_write(step.kv_c, step.k_pe, step.slots, cache, layout, k_scale=step.k_scale, gamma=step.gamma_kv,
                  eps=step.eps, rows=rows, flags=flags)
    torch.cuda.synchronize()
    assert torch.equal(cache, step.cache)
    assert int(flags) == 0
    # the rows handed on: normalised in FP64 and rounded (or, at a midpoint, to the other side), k_pe as it is
    x = O.bf16_bits_to_f64(inp["kv_c"])
    want = O.rmsnorm(x, O.bf16_bits_to_f64(inp["gamma_kv"]), float(np.float32(inp["eps"])))
    got = rows.double().cpu().numpy()
    assert (np.abs(got[:, :512] - want) <= (2.0 ** -8 + 2.0 ** -14) * np.abs(want)).all()
    assert torch.equal(rows[:, 512:], step.k_pe)
    step.close()


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("interleaved", [True, False])
def test_cache_write_with_rotation_and_without_norm(layout, interleaved):
    """Rotation in the pass gives the bytes of rotation before it; rows without gamma are quantised as they are."""
    rng = np.random.default_rng(layout)
    n, pages, page = 300, 30, 16
    kv, pe = bf16(rng, n, 512), bf16(rng, n, 64)
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64)).cuda()
    scale = torch.from_numpy(rng.uniform(0.01, 0.2, pages).astype(np.float32)).cuda()
    axis = rng.integers(0, 2, 32)
    axis[0] = 1
    pos = torch.from_numpy(rng.integers(0, 5000, (2, n)).astype(np.int32)).cuda()
    rot = R.Rotary(inv_freq(), axis, interleaved)
    a = torch.zeros(pages, page, C.ROW_BYTES[layout], dtype=torch.uint8, device="cuda")
    b, rows = a.clone(), torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    R.cache_write(kv, pe, slots, a, layout, k_scale=scale, rotary=rot, positions=pos, offset=3, rows=rows)
    turned = rot.apply(pe[:, None], pos, offset=3)[:, 0]
    R.cache_write(kv, turned, slots, b, layout, k_scale=scale)
    assert torch.equal(a, b)
    assert torch.equal(rows, torch.cat([kv, turned], 1))
    flat = a.view(-1, a.shape[2]).cpu().numpy()
    k64, p64 = kv.double().cpu().numpy(), turned.double().cpu().numpy()
    bits = turned.view(torch.int16).cpu().numpy().view(np.uint16)
    for t in range(0, n, 29):
        s = int(slots[t])
        if layout in (0, 3):
            ks = float(scale[s // page] if layout == 3 else scale[0])
            want = O.kv_row_e4m3(k64[t], p64[t], ks)
        elif layout == 1:
            want = O.kv_row_ds(k64[t], bits[t])[0]
        else:
            want = O.kv_row_nvfp4(k64[t], p64[t])[0]
        assert (flat[s] == want).all(), t


def test_cache_write_in_place_slots_beyond_the_cache_and_many_tokens():
    rng = np.random.default_rng(3)
    n, pages, page = 20000, 400, 64
    wide = bf16(rng, n, 2112)
    row = wide[:, 1536:]
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64)).cuda()
    slots[5], slots[6] = pages * page, 2 ** 40
    gamma = bf16(rng, 512)
    cache = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    apart = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    keep = wide[:, :1536].clone()
    R.cache_write(row[:, :512], row[:, 512:], slots, cache, 1, gamma=gamma, rows=apart, flags=flags)
    assert int(flags) == B.MLA_DEVERR_BAD_SLOT
    again = torch.zeros_like(cache)
    R.cache_write(row[:, :512], row[:, 512:], slots, again, 1, gamma=gamma, rows=row)
    assert torch.equal(row, apart) and torch.equal(wide[:, :1536], keep)
    assert torch.equal(cache, again)
    left = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    left[slots[slots < pages * page]] = False
    assert not cache.view(-1, 656)[left].any()


def test_cache_write_offsets_beyond_32_bits():
    """The last rows of a cache of more than 2^32 bytes."""
    rng = np.random.default_rng(4)
    page, pages = 64, 110000
    cache = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    kv, pe = bf16(rng, 4, 512), bf16(rng, 4, 64)
    slots = torch.tensor([pages * page - 1, 0, 2 ** 32 // 656 + 1, pages * page - 64], device="cuda")
    R.cache_write(kv, pe, slots, cache, 1)
    small = torch.zeros(1, 4, 656, dtype=torch.uint8, device="cuda")
    R.cache_write(kv, pe, torch.arange(4, device="cuda"), small, 1)
    assert torch.equal(cache.view(-1, 656)[slots], small[0])
    table = torch.tensor([[pages - 1], [(2 ** 32 // 656 + 1) // page]], dtype=torch.int32, device="cuda")
    rows = torch.empty(2, 576, dtype=torch.bfloat16, device="cuda")
    first = torch.tensor([63, (2 ** 32 // 656 + 1) % page], dtype=torch.int32, device="cuda")
    R.cache_read(cache, 1, None, table, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), rows, first=first)
    want = C.rows64(small[0].cpu().numpy()[[0, 2]], 1)
    assert (np.abs(rows.double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(want)).all()


# ---------------------------------------------------------------- cache_read


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("page", [1, 7, 64, 100])
@pytest.mark.parametrize("lens", [[1], [5, 0, 130, 1, 0], [700, 64, 65, 63] * 6, [12000, 3, 9000]])
def test_cache_read(layout, page, lens):
    rng = np.random.default_rng(layout * 10 + page)
    before = [n // 3 for n in lens]
    pages = sum(-(-n // page) for n in lens) + 3
    cache, k_scale = C.make_cache(rng, pages, page, layout)
    table = C.make_table(rng, lens, page, pages, width=max(1, max(-(-n // page) for n in lens)) + 2)
    count = [n - b for n, b in zip(lens, before)]
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    total = int(cu[-1])
    wide = torch.full((total + 5, 592), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = wide[:, :576]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.cache_read(torch.from_numpy(cache).cuda(), layout, torch.from_numpy(k_scale).cuda(), torch.from_numpy(table).cuda(),
                 torch.from_numpy(cu).cuda(), rows, first=torch.tensor(before, dtype=torch.int32, device="cuda"),
                 flags=flags)
    assert int(flags) == 0
    assert (wide[:, 576:] == 7.0).all() and (wide[total:] == 7.0).all()
    p, o = [], []
    for r, n in enumerate(lens):
        for i in range(before[r], n):
            p.append(table[r, i // page])
            o.append(i % page)
    p, o = np.array(p, dtype=int), np.array(o, dtype=int)
    sc = (k_scale[p] if layout == 3 else np.repeat(k_scale[:1], len(p))).astype(np.float64)
    want = C.rows64(cache[p, o], layout, sc)
    err = np.abs(rows[:total].double().cpu().numpy() - want)
    assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want) + 1e-38).all()


def test_cache_read_absent_pages_and_short_outputs():
    rng = np.random.default_rng(9)
    page, pages = 16, 8
    cache, k_scale = C.make_cache(rng, pages, page, 0)
    cache_t, scale = torch.from_numpy(cache).cuda(), torch.from_numpy(k_scale).cuda()
    table = torch.tensor([[0, -1, 2], [3, 8, 5]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([2, 50, 110], dtype=torch.int32, device="cuda")  # rows 0, 1 are no request's
    rows = torch.full((100, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.cache_read(cache_t, 0, scale, table, cu, rows, first=torch.tensor([0, -2], dtype=torch.int32, device="cuda"),
                 flags=flags)
    assert int(flags) == B.MLA_DEVERR_BAD_SLOT
    assert (rows[:2] == 3.0).all()
    assert (rows[2 + 16:2 + 32] == 0).all()  # an absent page
    assert (rows[50:52] == 0).all()  # before the first position
    assert (rows[52 + 16:52 + 32] == 0).all()  # a page beyond the cache
    want = C.rows64(cache[3], 0, k_scale)
    got = rows[52:68].double().cpu().numpy()
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
    got = rows[84:100].double().cpu().numpy()
    want = C.rows64(cache[5], 0, k_scale)
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()


def test_row_operators_in_a_graph_and_on_another_stream():
    """Captured once, replayed on new inputs: what was read is what was written."""
    rng = np.random.default_rng(11)
    n, pages, page = 70, 4, 32
    kv, pe, pos = bf16(rng, n, 512), bf16(rng, n, 64), torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, device="cuda")
    cache = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rows, back = (torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rot = R.Rotary(inv_freq())
    side = torch.cuda.Stream()

    def step():
        R.cache_write(kv, pe, slots, cache, 1, rotary=rot, positions=pos, rows=rows)
        R.cache_read(cache, 1, None, table, cu, back)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = back.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rot.close()  # (a captured call keeps what it needs)
    kv.copy_(bf16(rng, n, 512))
    pos += 500
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first, back)
    assert torch.equal(back[:, 512:], rows[:, 512:])  # k_pe is kept in BF16
    scale = kv.float().view(n, 4, 128).abs().amax(2).repeat_interleave(128, 1)
    assert ((back[:, :512].float() - kv.float()).abs() <= (2.0 ** -4 * kv.float().abs()).maximum(scale * 2.0 ** -16)).all()
