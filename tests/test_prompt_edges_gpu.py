"""The prompt's operators at the ends of what they take.

Rows of the cache are compared byte by byte; tolerances of attention are those of
test_prompt_attn_gpu (derived there).
"""

import numpy as np
import pytest
import torch

from mla_query_projection_gb300 import binding as B
from mla_query_projection_gb300 import runner as R

from .test_prompt_attn_gpu import cuda_device  # noqa: F401
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
