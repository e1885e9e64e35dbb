"""Attention of packed documents on the GPU against its plain 64-bit form.

Tolerances, derived before the first run.
 * scores: the products of BF16 values are exact in FP32; a sum of 192 of them is
   off by at most 192 * 2^-23 of X = scale * sum |q_c k_c| (2^-23: tensor cores may
   cut where others round) < 2^-15.4 X; scaling and the reference add 2^-22 of the
   score.  Capped: 2^-20 of the cap more; a bias: 2^-22 of it.
 * weights: the exponential and the sums add 2^-20 relative; BF16 2^-8.
 * so with A = sum p |v|: |out error| <= (2^-8 + 2 e) A + 2^-8 |out|, and the
   logarithm of the sum is off by at most e + 2^-22 |lse|, e the score's bound
   plus 2^-20.
"""

import math

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def cuda_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()
    torch.cuda.set_device(0)
    yield


def seen_by(nq, nk, causal, prefix, device="cuda"):
    j, place = torch.arange(nk, device=device), torch.arange(nq, device=device)[:, None] + nk - nq
    return ((j <= place) | (j < prefix)) if causal else torch.ones(nq, nk, dtype=torch.bool, device=device)


def document64(q, k, k_pe, v, causal, prefix, scale, cap, slopes):
    """(out, lse, A, score bound) of one document: q [nq, h, 192], k, v [nk, h, 128], k_pe [nk, 64], FP64.
    Values that a row does not see are not used (they may be anything)."""
    nq, nk, heads = len(q), len(k), q.shape[1]
    dev = q.device
    out = torch.zeros(nq, heads, 128, dtype=torch.float64, device=dev)
    lse = torch.full((nq, heads), -math.inf, dtype=torch.float64, device=dev)
    mass, slack = torch.zeros_like(out), torch.zeros_like(lse)
    if nq == 0 or nk == 0:
        return out, lse, mass, slack
    seen = seen_by(nq, nk, causal, prefix, dev)
    place = torch.arange(nq, device=dev)[:, None] + nk - nq
    far = (place - torch.arange(nk, device=dev)).abs().double()
    for h in range(heads):
        key = torch.cat([k[:, h], k_pe], 1)
        x = q[:, h] @ key.T * scale
        mag = torch.where(seen, q[:, h].abs() @ key.abs().T * scale, 0.0).amax(1)
        if cap:
            x = cap * torch.tanh(x / cap)
        if slopes is not None:
            x = x - slopes[h] * far
        big = torch.where(seen, x.abs(), 0.0).amax(1)
        x = torch.where(seen, x, -math.inf)
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        tot = p.sum(1, keepdim=True)
        p = p / torch.where(tot == 0, 1.0, tot)
        fine = torch.isfinite(v[:, h])
        vv = torch.where(fine, v[:, h], 0.0)
        out[:, h] = p @ vv
        if not fine.all():  # what is not finite reaches the rows that see it
            for j, c in (~fine).nonzero().tolist():
                out[seen[:, j], h, c] += v[j, h, c]
        mass[:, h] = p @ vv.abs()
        lse[:, h] = (m + torch.log(tot))[:, 0]
        bias = 0.0 if slopes is None else float(abs(slopes[h])) * far.max()
        slack[:, h] = 2.0 ** -15.4 * mag + 2.0 ** -22 * (big + bias) + 2.0 ** -20 * (1 + cap)
    return out, lse, mass, slack


def inputs(seed, tq, tk, heads, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return ((r(tq, heads, 192) * std).to(torch.bfloat16), r(tk, heads, 256).to(torch.bfloat16),
            r(tk, 64).to(torch.bfloat16))


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def check(got, lse, want, label):
    o, z, mass, slack = want
    got, lse = got.double(), lse.double()
    none = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), none), label
    assert (got[none] == 0).all(), label
    err = (lse - z)[~none].abs()
    assert (err <= (slack + 2.0 ** -22 * z.abs())[~none]).all(), (label, "lse", float((err / slack[~none]).max()))
    odd = ~torch.isfinite(o)
    assert torch.equal(torch.isnan(got), torch.isnan(o)), label
    assert torch.equal(got[odd & ~torch.isnan(o)], o[odd & ~torch.isnan(o)]), label
    bound = (2.0 ** -8 + 2 * slack)[..., None] * mass + 2.0 ** -8 * o.abs() + 1e-30
    err = torch.where(odd, 0.0, (got - o).abs())
    bound = torch.where(odd, 1.0, bound)
    assert (err <= bound).all(), (label, "out", float((err / bound).max()))


def attend(seed, docs, heads, causal=True, prefix=None, cap=0.0, slopes=None, pad=0, change=None, attn=None, scale=SCALE):
    """docs: (queries, keys) of each document; every row is checked."""
    nq, nk = [d[0] for d in docs], [d[1] for d in docs]
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    tq, tk = int(cu_q[-1]) + pad, int(cu_k[-1])
    q, kv, k_pe = inputs(seed, tq, tk, heads)
    if change is not None:
        change(q, kv, k_pe)
    s = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    out = torch.full((tq, heads, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq, heads), 5.0, device="cuda")
    own = attn is None
    attn = attn or R.PromptAttention(heads)
    attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32(cu_q), scale, cu_k=i32(cu_k),
                causal=causal, prefix=None if prefix is None else i32(prefix), softcap=cap, slopes=s, out=out, lse=lse)
    flags = attn.error_flags()
    assert flags == 0, hex(flags)
    if own:
        attn.close()
    if pad:
        assert (out[-pad:] == 5.0).all() and (lse[-pad:] == 5.0).all()
    for d in range(len(docs)):
        a, b, c, e = cu_q[d], cu_q[d + 1], cu_k[d], cu_k[d + 1]
        want = document64(q[a:b].double(), kv[c:e, :, :128].double(), k_pe[c:e].double(), kv[c:e, :, 128:].double(), causal,
                          0 if prefix is None else prefix[d], scale, cap, None if s is None else s.double())
        check(out[a:b], lse[a:b], want, (d, docs[d], heads, causal, cap))
    return out, lse


@pytest.mark.parametrize("heads", [1, 3, 16])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 500, 1000])
def test_one_document(n, heads):
    attend(n, [(n, n)], heads)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("docs", [[(1, 1)] * 70, [(5, 5), (300, 300), (0, 0), (128, 128), (1, 1), (257, 257)],
                                  [(10, 500), (500, 10), (130, 0), (0, 40), (256, 255), (1, 2000)],
                                  [(200 + 7 * i, 200 + 7 * i) for i in range(12)]])
def test_packed_documents(docs, causal):
    attend(len(docs), docs, 5, causal=causal, pad=3)


@pytest.mark.parametrize("cap,slopes,prefix", [(30.0, False, False), (0.0, True, False), (0.0, False, True), (5.0, True, True),
                                               (1000.0, False, True), (1e-3, False, False)])
@pytest.mark.parametrize("causal", [True, False])
def test_caps_biases_and_prefixes(cap, slopes, prefix, causal):
    docs = [(300, 300), (17, 400), (400, 390), (1, 1), (129, 1000)]
    attend(3, docs, 4, causal=causal, cap=cap, slopes=[0.5, 2.0 ** -8, 0.0, -0.01] if slopes else None,
           prefix=[100, 395, 0, 1, 5000] if prefix else None)


@pytest.mark.parametrize("nq,nk,heads",
                         [(1, 1, 2), (1, 5000, 1), (3, 20000, 16), (200, 9000, 2), (300, 4000, 7)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_few_rows_over_many_keys(nq, nk, heads, cap):
    """Keys split over several workers, whose sums are joined."""
    attend(nk, [(nq, nk)], heads, cap=cap)


def test_split_documents_of_very_different_lengths():
    attend(21, [(1, 9000), (1, 3), (2, 0), (1, 700), (1, 1)], 2, pad=4)
    attend(22, [(1, 9000), (4, 3), (2, 0), (1, 700)], 2, causal=False)


def test_long_document():
    attend(7, [(4100, 4100)], 2)


def test_rows_whose_maximum_keeps_growing():
    """Every key tile's scores are far above the last one's: the reference moves in each."""
    def change(q, kv, k_pe):
        q[..., 0] = 8.0
        kv[:, :, 0] = (torch.arange(len(kv), device="cuda").float() / 8).to(torch.bfloat16)[:, None]

    attend(8, [(700, 700)], 3, change=change)
    attend(8, [(2, 6000)], 3, change=change)  # over split keys too


def test_large_and_tiny_scores():
    for factor in (1e-3, 30.0):
        attend(9, [(300, 300)], 2, change=lambda q, kv, k_pe: q.mul_(factor))
    attend(9, [(300, 300)], 2, scale=0.0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,at,splits", [(300, 260, False), (256, 255, False), (900, 500, False), (9000, 8990, True)])
def test_values_that_are_not_seen_may_be_anything(bad, n, at, splits):
    """An infinity or a NaN in a value reaches the rows that see its key, and no others; neither do those of other
    documents."""
    nq = 40 if splits else n

    def change(q, kv, k_pe):
        kv[at + 3, 1, 128 + 77] = bad
        kv[at + 3, 0, 128 + 5] = bad
        kv[at + 5, 0, 128 + 5] = -bad  # opposite infinities: NaN where both are seen
        kv[n + 3:, :, 128:] = bad  # the next document
        kv[n + 3:, :, :128] = bad
        kv[:3, :, :] = bad  # and the one before

    docs = [(3, 3), (nq, n), (70, 70)]
    nqs, nks = zip(*docs)
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nqs)]), np.concatenate([[0], np.cumsum(nks)])
    q, kv, k_pe = inputs(5, int(cu_q[-1]), int(cu_k[-1]), 2)
    change(q, kv, k_pe)
    attn = R.PromptAttention(2)
    lse = torch.zeros(len(q), 2, device="cuda")
    out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32(cu_q), SCALE, cu_k=i32(cu_k),
                         lse=lse)
    assert attn.error_flags() == 0
    a, b, c, e = cu_q[1], cu_q[2], cu_k[1], cu_k[2]
    want = document64(q[a:b].double(), kv[c:e, :, :128].double(), k_pe[c:e].double(), kv[c:e, :, 128:].double(), True, 0,
                      SCALE, 0.0, None)
    check(out[a:b], lse[a:b], want, (bad, n, at))
    attn.close()


@pytest.mark.parametrize("docs", [
    [(200, 50), (3, 3)] * 20 + [(256, 256), (7, 7), (500, 500)],  # whose first 128 rows see nothing, again and again
    [(1, 1), (300, 20)] * 15 + [(140, 140), (2, 2)] * 8,
    [(40, 9000), (64, 64), (1, 3000), (5, 5)],  # split keys
    [(130, 300), (130, 131), (1, 129), (257, 100)] * 6,
])
def test_documents_beside_others_that_are_not_finite(docs):
    """Every second document is NaN all over: the others' rows are as without it."""
    heads = 6
    nq, nk = zip(*docs)
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    q, kv, k_pe = inputs(16, int(cu_q[-1]), int(cu_k[-1]), heads)
    for d in range(1, len(docs), 2):
        kv[cu_k[d]:cu_k[d + 1]] = math.nan
        k_pe[cu_k[d]:cu_k[d + 1]] = math.nan
        q[cu_q[d]:cu_q[d + 1]] = math.nan
    attn = R.PromptAttention(heads)
    lse = torch.zeros(len(q), heads, device="cuda")
    for causal in (True, False):
        for _ in range(3):
            out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32(cu_q), SCALE, cu_k=i32(cu_k),
                                 causal=causal, lse=lse)
            assert attn.error_flags() == 0
            for d in range(0, len(docs), 2):
                a, b, c, e = cu_q[d], cu_q[d + 1], cu_k[d], cu_k[d + 1]
                want = document64(q[a:b].double(), kv[c:e, :, :128].double(), k_pe[c:e].double(), kv[c:e, :, 128:].double(),
                                  causal, 0, SCALE, 0.0, None)
                check(out[a:b], lse[a:b], want, (d, docs[d], causal))
    attn.close()


def test_keys_and_queries_that_are_not_finite():
    """A NaN key that a row does not see leaves it alone; a NaN query makes its own row NaN."""
    q, kv, k_pe = inputs(6, 200, 200, 2)
    kv[150, :, 3] = math.nan
    q[20, 1, 5] = math.nan
    attn = R.PromptAttention(2)
    lse = torch.zeros(200, 2, device="cuda")
    out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 200]), SCALE, lse=lse)
    assert torch.isnan(out[150:]).all() and torch.isnan(out[20, 1]).all() and torch.isnan(lse[20, 1])
    sound = torch.ones(200, 2, dtype=torch.bool, device="cuda")
    sound[150:], sound[20, 1] = False, False
    assert torch.isfinite(out[sound]).all() and torch.isfinite(lse[sound]).all()
    attn.close()


def test_strides_orders_and_alignment():
    """Head-major queries, wider rows, contiguous parts, a strided output: the same bits."""
    tq, tk, heads = 150, 333, 6
    q, kv, k_pe = inputs(10, tq, tk, heads)
    attn = R.PromptAttention(heads)
    cu = dict(cu_q=i32([0, 100, tq]), cu_k=i32([0, 200, tk]))
    base, lse = torch.empty(tq, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(tq, heads, device="cuda")
    attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], softmax_scale=SCALE, out=base, lse=lse, **cu)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)  # [heads][tokens][192]
    kvh = torch.empty(heads, tk, 264, dtype=torch.bfloat16, device="cuda")
    kvh[..., :256] = kv.transpose(0, 1)
    kvh = kvh.transpose(0, 1)
    pe = torch.zeros(tk, 2112, dtype=torch.bfloat16, device="cuda")
    pe[:, 2048:] = k_pe
    out = torch.zeros(heads, tq, 136, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    attn.attend(qh[..., :128], qh[..., 128:].contiguous(), kvh[..., :128], pe[:, 2048:], kvh[..., 128:256], softmax_scale=SCALE,
                out=out[..., :128], **cu)
    assert torch.equal(out[..., :128], base) and not out[..., 128:].any()
    got, none = attn.attend(q[..., :128].contiguous(), q[..., 128:], kv[..., :128].contiguous(), k_pe, kv[..., 128:],
                            softmax_scale=SCALE, **cu)
    assert none is None and torch.equal(got, base)
    assert attn.error_flags() == 0
    attn.close()


def test_cu_beyond_the_tensors_is_flagged_and_cut():
    q, kv, k_pe = inputs(11, 100, 100, 2)
    attn = R.PromptAttention(2)
    out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 40, 130]), SCALE)
    assert attn.error_flags() == B.MLA_DEVERR_BAD_SLOT
    want, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 40, 100]), SCALE)
    assert attn.error_flags() == 0
    assert torch.equal(out, want)
    for odd in ([0, 60, 30], [0, 100] * 40, [-5, 50, 100], [2 ** 31 - 1, -2 ** 31, 7]):
        attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32(odd), SCALE)
        assert attn.error_flags() == B.MLA_DEVERR_BAD_SLOT
    again, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 40, 100]), SCALE)
    assert attn.error_flags() == 0 and torch.equal(again, want)
    attn.close()


def test_no_rows_no_keys():
    q, kv, k_pe = inputs(12, 5, 5, 2)
    attn = R.PromptAttention(2)
    out, _ = attn.attend(q[:0, :, :128], q[:0, :, 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 0]), SCALE,
                         cu_k=i32([0, 5]))
    assert out.shape == (0, 2, 128)
    lse = torch.zeros(5, 2, device="cuda")
    out, _ = attn.attend(q[..., :128], q[..., 128:], kv[:0, :, :128], k_pe[:0], kv[:0, :, 128:], i32([0, 5]), SCALE,
                         cu_k=i32([0, 0]), lse=lse)
    assert not out.any() and torch.isneginf(lse).all()
    assert attn.error_flags() == 0
    attn.close()


def test_refusals_of_a_live_handle():
    q, kv, k_pe = inputs(13, 8, 8, 4)
    attn = R.PromptAttention(4)
    cu = i32([0, 8])
    good = dict(q_nope=q[..., :128], q_pe=q[..., 128:], k_nope=kv[..., :128], k_pe=k_pe, v=kv[..., 128:], cu_q=cu,
                softmax_scale=SCALE)
    out = torch.empty(8, 4, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q_nope=q[:, :3, :128]), dict(q_nope=q[..., :127]), dict(q_pe=q[..., 128:191]), dict(q_pe=q[:7, :, 128:]),
                dict(k_nope=kv[:7, :, :128]), dict(k_pe=k_pe[:7]), dict(k_pe=k_pe[:, :63]), dict(v=kv[..., 129:]),
                dict(v=kv[..., 128:].float()), dict(cu_q=cu.long()), dict(cu_q=cu[:1]), dict(cu_k=cu[:1]), dict(prefix=cu[:0]),
                dict(softmax_scale=-1.0), dict(softmax_scale=math.nan), dict(softmax_scale="x"), dict(softcap=-1.0),
                dict(softcap=math.inf), dict(softcap=1001.0), dict(softcap=1e-7), dict(slopes=torch.zeros(3, device="cuda")), dict(out=out[:7]),
                dict(out=torch.empty(8, 1, 128, dtype=torch.bfloat16, device="cuda").expand(8, 4, 128)),
                dict(out=torch.empty(8 * 132 + 4 * 128, dtype=torch.bfloat16, device="cuda").as_strided((8, 4, 128), (136, 128, 1))),
                dict(lse=torch.empty(8, 3, device="cuda")), dict(q_nope=q.cpu()[..., :128]),
                dict(q_nope=torch.empty(8, 4, 130, dtype=torch.bfloat16, device="cuda")[..., 1:129])):
        with pytest.raises(B.MlaError):
            attn.attend(**{**good, **bad})
    attn.close()
    with pytest.raises(B.MlaError, match="closed"):
        attn.attend(**good)


def test_graph_replays_streams_and_two_handles():
    """Captured, replayed on new inputs, beside another handle's calls on another stream: the same bits as alone."""
    heads = 3
    shapes = [([(1, 4000), (2, 300)], 0), ([(400, 400)], 1)]
    attns = [R.PromptAttention(heads) for _ in shapes]
    data, outs, graphs = [], [], []
    for (docs, _), attn in zip(shapes, attns):
        nq, nk = zip(*docs)
        cu = [i32(np.concatenate([[0], np.cumsum(x)])) for x in (nq, nk)]
        q, kv, k_pe = inputs(14, sum(nq), sum(nk), heads)
        out = torch.zeros(sum(nq), heads, 128, dtype=torch.bfloat16, device="cuda")
        data.append((q, kv, k_pe, cu))
        outs.append(out)

        def call(q=q, kv=kv, k_pe=k_pe, cu=cu, out=out, attn=attn):
            attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu[0], SCALE, cu_k=cu[1], out=out)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, call))
    for q, kv, k_pe, _ in data:
        q.neg_()
        kv.mul_(0.5)
    want = []
    for (_, call), out in zip(graphs, outs):
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, out, w in zip(attns, outs, want):
        assert torch.equal(out, w)
        assert a.error_flags() == 0
        a.close()


def test_output_belongs_to_the_calls_stream():
    q, kv, k_pe = inputs(15, 64, 64, 2)
    attn, s = R.PromptAttention(2), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, 64]), SCALE)
    torch.cuda.synchronize()
    out, _ = attn.attend(*args, stream=s)
    with torch.cuda.stream(s):
        here = torch.empty(64, 2, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    want, _ = attn.attend(*args)
    assert torch.equal(out, want)
    assert here.data_ptr() != out.data_ptr()
    attn.close()


def test_a_prompt_in_chunks_and_its_first_decoded_token():
    """The layer's path together: tables, rotated queries, cache rows, the context read back, the up-projection, prompt
    attention; the last token's output agrees with latent attention over the same cache."""
    rng = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, std=1.0: (torch.randn(s, generator=rng, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    heads, page, pages, width = 4, 16, 64, 40
    lens, table = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pages, dtype=torch.int32, device="cuda"), i32([pages])
    w_uk, w_uv = r(heads, 128, 512, std=0.05), r(heads, 128, 512, std=0.05)
    gamma = r(512, std=0.1) + 1
    cache = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
    rot = R.Rotary(10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64))
    attn, latent = R.PromptAttention(heads), R.PagedAttention(16, heads)
    flags = i32([0])
    for new in ([100, 37, 5], [60, 0, 130]):
        n, before = sum(new), lens.clone()
        slots = torch.empty(n + 2, dtype=torch.int64, device="cuda")
        row, tlen, cu_q = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (n + 2, n + 2, 4))
        R.tables_step(i32(new), lens, table, free, count, page, lens, count, slots, row, tlen, cu_q, flags)
        kv_row, q = r(n + 2, 2112), r(n + 2, heads, 192)
        R.cache_write(kv_row[:, 1536:2048], kv_row[:, 2048:], slots, cache, 1, gamma=gamma, rotary=rot, positions=tlen,
                      offset=-1, flags=flags)
        rot.apply(q[..., 128:], tlen, out=q[..., 128:], offset=-1)
        cu_k = torch.cat([i32([0]), lens.cumsum(0, dtype=torch.int32)])
        keys = torch.empty(int(cu_k[-1]), 576, dtype=torch.bfloat16, device="cuda")
        R.cache_read(cache, 1, None, table, cu_k, keys, flags=flags)
        up = torch.einsum("tc,hpc->thp", keys[:, :512].float(), torch.cat([w_uk, w_uv], 1).float()).to(torch.bfloat16)
        lse = torch.zeros(n + 2, heads, device="cuda")
        out, _ = attn.attend(q[..., :128], q[..., 128:], up[..., :128], keys[:, 512:], up[..., 128:], cu_q, SCALE, cu_k=cu_k,
                             lse=lse)
        assert int(flags) == 0 and attn.error_flags() == 0
        for d, k in enumerate(new):
            if not k:
                continue
            a, b, c, e = int(cu_q[d]), int(cu_q[d + 1]), int(cu_k[d]), int(cu_k[d + 1])
            want = document64(q[a:b].double(), up[c:e, :, :128].double(), keys[c:e, 512:].double(), up[c:e, :, 128:].double(),
                              True, 0, SCALE, 0.0, None)
            check(out[a:b], lse[a:b], want, (new, d))
            # the last token through the latent space: q absorbed, 512-wide values, W_UV behind
            t = b - 1
            ql = torch.einsum("hp,hpc->hc", q[t, :, :128].float(), w_uk.float()).to(torch.bfloat16)
            lo, _ = latent.decode(ql[None], q[t:t + 1, :, 128:], cache, 1, table[d:d + 1], lens[d:d + 1], SCALE)
            got = torch.einsum("hc,hvc->hv", lo[0].double(), w_uv.double())
            # q_latent, the keys, the values and the weights are rounded on one side or the other: 2^-8 each, and the
            # decode's weights 2^-6.5; scores of size s turn 2 * 2^-8 of it into weights
            up64 = torch.einsum("tc,hpc->thp", keys[c:e, :512].double(), w_uv.double())
            x = torch.einsum("hp,thp->ht", q[t, :, :128].double().abs(), up[c:e, :, :128].double().abs()) * SCALE
            rough = (2.0 ** -6.5 + 3 * 2.0 ** -8 + 4 * 2.0 ** -8 * float(x.max())) * up64.abs().amax(0)
            assert ((got - out[t].double()).abs() <= rough).all()
    for a in (attn, latent):
        a.close()


def test_steep_slopes_near_the_row():
    """A slope of 3,000 leaves a row its own key alone (the next weighs e^-3000 times more
    than any score here, |x| < 100).  Its own distance is zero, so the bias has nothing to
    be rounded: the logarithm of the sum is its score, off by the score's bound alone (the
    sum of 192 products and its scaling), not by 2^-24 of slope times place."""
    n, heads = 700, 2
    q, kv, k_pe = inputs(31, n, n, heads)
    attn = R.PromptAttention(heads)
    lse = torch.empty(n, heads, device="cuda")
    cu = i32([0, n])
    out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu, SCALE,
                         slopes=torch.full((heads,), 3000.0, device="cuda"), lse=lse)
    attn.close()
    key = torch.cat([kv[..., :128], k_pe[:, None].expand(n, heads, 64)], -1).double()
    score = (q.double() * key).sum(-1) * SCALE
    mag = (q.double() * key).abs().sum(-1) * SCALE
    assert ((lse.double() - score).abs() <= 2.0 ** -15.4 * mag + 2.0 ** -21 * (1 + score.abs())).all()
    assert torch.equal(out, kv[..., 128:])


@pytest.mark.parametrize("seed,causal,prefix,cap,bias", [(1, True, False, 0.0, False), (2, True, True, 0.0, False),
                                                         (3, False, False, 0.0, False), (4, True, False, 30.0, False),
                                                         (5, True, True, 0.0, True), (6, True, True, 20.0, True)])
def test_many_items_of_all_kinds_one_after_another(seed, causal, prefix, cap, bias):
    """Fifty items a worker: one query tile or two, one key tile or several, rows before all
    keys, documents without rows or without keys, in random order."""
    rng = np.random.default_rng(seed)
    docs = []
    for _ in range(45):
        nq = int(rng.choice([0, 1, 5, 64, 127, 128, 129, 200, 255, 256, 257, 300, 400]))
        more = int(rng.choice([0, 0, 0, 1, 100, 128, 300, -1, -100, -1000]))
        docs.append((nq, max(0, nq + more)))
    attend(seed, docs, 128, causal=causal, prefix=[int(x) for x in rng.integers(0, 300, 45)] if prefix else None, cap=cap,
           slopes=[float(2.0 ** -(1 + h % 8)) for h in range(128)] if bias else None, pad=2)


def test_the_order_of_the_work_does_not_show():
    """Items go to whichever worker is free: calls alike give the same bytes."""
    rng = np.random.default_rng(12)
    n = [int(x) for x in rng.choice([1, 60, 128, 130, 250, 300, 513], 20)]
    heads, cu = 96, np.concatenate([[0], np.cumsum(n)])
    q, kv, k_pe = inputs(12, int(cu[-1]), int(cu[-1]), heads)
    attn, where = R.PromptAttention(heads), i32(cu)
    got = []
    for _ in range(6):
        lse = torch.empty(len(q), heads, device="cuda")
        out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], where, SCALE, softcap=25.0, lse=lse)
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    attn.close()
