"""The prompt's operators at the ends of what they take.

Rows of the cache are compared byte by byte; tolerances of attention are those of
test_prompt_attn_gpu (derived there).
"""

import math

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

from .test_prompt_attn_gpu import SCALE, attend, cuda_device, i32, inputs  # noqa: F401
from .test_prompt_rows_gpu import write_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [0, 1, 2, 3])
@pytest.mark.parametrize("norm", [True, False])
def test_zeros_keep_their_sign_in_the_cache(layout, norm):
    """Zeros of either sign in kv_c and k_pe, and in gamma: the decode step's bytes; where
    rows are not normalised, the codes of zeros are 0x00 and 0x80."""
    inp = write_case(layout, 70, seed=layout)
    rng = np.random.default_rng(layout)
    for x in (inp["kv_c"], inp["k_pe"]):
        x[rng.random(x.shape) < 0.1] = 0x8000
        x[rng.random(x.shape) < 0.1] = 0
    inp["gamma_kv"][3::11], inp["gamma_kv"][5::13] = 0, 0x8000
    step = R.DecodeStep(inp)
    cache = step.cache.clone()
    if norm:
        assert step.decode() == B.MLA_OK
        R.cache_write(step.kv_c, step.k_pe, step.slots, cache, layout, k_scale=step.k_scale, gamma=step.gamma_kv, eps=step.eps)
        assert torch.equal(cache, step.cache)
    else:
        R.cache_write(step.kv_c, step.k_pe, step.slots, cache, layout, k_scale=step.k_scale)
        # where the codes of one byte a value lie in a row: of the latent part, of the rope part
        at = {0: (0, 512), 1: (0, None), 2: (None, 288), 3: (0, 512)}[layout]
        flat = cache.view(-1, cache.shape[2])
        keep = step.slots >= 0
        for part, x in zip(at, (step.kv_c, step.k_pe)):
            if part is None:
                continue
            codes = flat[step.slots[keep], part:part + x.shape[1]]
            zero = x[keep] == 0
            want = torch.where(torch.signbit(x[keep].float()), 0x80, 0x00)
            assert torch.equal(codes[zero].int(), want[zero].int())
    step.close()


# ---------------------------------------------------------------- attention


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("causal,prefix", [(True, None), (True, 700), (False, None)])
@pytest.mark.parametrize("cap", [15.0, 400.0])
def test_long_capped_documents(cap, causal, prefix, slopes):
    """Whole query tiles over 2,000 keys and more that are not split: capped scores are taken
    64 columns at a time, with and without biases, on the diagonal, in a prefix, on both sides."""
    heads = 16
    attend(41, [(2117, 2117)], heads, causal=causal, prefix=None if prefix is None else [prefix], cap=cap,
           slopes=[0.3 * 2.0 ** -h for h in range(heads)] if slopes else None)


@pytest.mark.parametrize("slopes", [False, True])
def test_long_capped_documents_of_ragged_lengths(slopes):
    docs = [(2500, 2500), (130, 2700), (1900, 1800), (257, 2300)]
    attend(42, docs, 5, prefix=[0, 2650, 40, 1], cap=25.0, slopes=[0.2, -0.01, 0.0, 2.0 ** -7, 1.0] if slopes else None)


@pytest.mark.parametrize("nq,nk,heads", [(3, 20000, 16), (300, 4000, 7), (129, 5000, 3)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("causal,prefix", [(True, None), (True, 1500), (False, None)])
def test_split_keys_with_biases_and_prefixes(nq, nk, heads, cap, causal, prefix):
    attend(nk, [(nq, nk)], heads, causal=causal, prefix=None if prefix is None else [nk - nq + 20 if nq > 128 else prefix],
           cap=cap, slopes=[0.05 * 2.0 ** -h for h in range(heads)])


@pytest.mark.parametrize("docs,heads", [([(700, 700)], 3), ([(100, 900)], 2), ([(2, 6000)], 3), ([(260, 3000)], 4)])
@pytest.mark.parametrize("cap", [0.0, 900.0])
def test_references_that_move_with_every_key_tile(docs, heads, cap):
    """Scores rise by 16 * 16 * 192^-0.5 = 18.5 a key tile, 26.6 in base 2: further than a
    reference may lie below them, in every tile."""
    def change(q, kv, k_pe):
        q[..., 0] = 16.0
        kv[:, :, 0] = (torch.arange(len(kv), device="cuda").float() / 8).to(torch.bfloat16)[:, None]

    attend(43, docs, heads, cap=cap, change=change)


@pytest.mark.parametrize("docs,heads", [([(1000, 1000)], 3), ([(90, 1000)], 3), ([(2, 9000)], 3), ([(300, 4000)], 3),
                                        ([(700, 700), (40, 650), (650, 700)], 3)])
@pytest.mark.parametrize("how", ["steep", "wide", "cap", "all"])
def test_an_infinite_value_counts_whatever_its_weight(docs, heads, how):
    """Keys that a row sees with a weight that underflows, in tiles on an edge and within: an
    infinity is an infinity, infinities of both signs and NaN are NaN, in every row that sees them."""
    def change(q, kv, k_pe):
        if how == "wide":
            q.mul_(60.0)
        at = 0
        for _, nk in docs:
            for key, column, bad in ((100, 7, math.inf), (300, 9, -math.inf), (100, 11, math.inf), (300, 11, -math.inf),
                                     (600, 13, math.nan), (639, 127, math.inf)):
                kv[at + key, :, 128 + column] = bad
            at += nk

    attend(46, docs, heads, causal=how != "all", cap=30.0 if how == "cap" else 0.0,
           slopes=None if how == "wide" else [3000.0, 20.0, 0.5], change=change)


@pytest.mark.parametrize("docs,heads", [([(700, 700)], 3), ([(100, 1500)], 2), ([(2, 9000)], 3), ([(260, 4000)], 4),
                                        ([(40, 40), (300, 300)], 2)])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("signs", [False, True])
def test_values_up_to_the_end_of_the_range(docs, heads, rising, signs):
    """Values of 2^126: a thousand of them are beyond FP32, their average is not.  With scores
    that rise a weight is taken relative to one far below it."""
    def change(q, kv, k_pe):
        v = kv[..., 128:].float().clamp(-1, 1)
        kv[..., 128:] = ((v if signs else 0.5 + 0.5 * v.abs()) * 2.0 ** 126).to(torch.bfloat16)
        if rising:
            q[..., 0] = 7.0
            kv[:, :, 0] = (torch.arange(len(kv), device="cuda").float() / 8).to(torch.bfloat16)[:, None]

    attend(44, docs, heads, change=change)
    attend(44, docs, heads, change=change, causal=False)


@pytest.mark.parametrize("docs,heads", [([(700, 700)], 3), ([(3, 20000)], 16)])
def test_small_values(docs, heads):
    """Values of 2^-85, far above what the tolerance adds (2^-99.6)."""
    attend(45, docs, heads, change=lambda q, kv, k_pe: kv[..., 128:].mul_(2.0 ** -85))


@pytest.mark.parametrize("slope", [1e5, 1e8, 1e31, 1e36, 3e38])
@pytest.mark.parametrize("n,nq", [(700, 700), (827, 700), (9000, 3)])
def test_slopes_up_to_the_end_of_the_range(slope, n, nq):
    """Any key but a row's own has a weight of zero, its bias finite or not; the own one, at no
    distance, has no bias (see test_steep_slopes_near_the_row)."""
    heads = 2
    q, kv, k_pe = inputs(47, nq, n, heads)
    attn = R.PromptAttention(heads)
    lse = torch.empty(nq, heads, device="cuda")
    for cap in (0.0, 30.0):
        out, _ = attn.attend(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], i32([0, nq]), SCALE,
                             cu_k=i32([0, n]), softcap=cap, slopes=torch.full((heads,), slope, device="cuda"), lse=lse)
        key = torch.cat([kv[..., :128], k_pe[:, None].expand(n, heads, 64)], -1).double()[n - nq:]
        score = (q.double() * key).sum(-1) * SCALE
        mag = (q.double() * key).abs().sum(-1) * SCALE
        score = cap * torch.tanh(score / cap) if cap else score
        assert ((lse.double() - score).abs() <= 2.0 ** -15.4 * mag + 2.0 ** -20 * (1 + cap) + 2.0 ** -21 * score.abs()).all()
        assert torch.equal(out, kv[n - nq:, :, 128:])
    assert attn.error_flags() == 0
    attn.close()


def test_the_largest_scale():
    """Scores of zero stay zero."""
    attend(48, [(300, 300)], 2, scale=2.9e38, change=lambda q, kv, k_pe: q.zero_())
