"""Token log probabilities of many rows in one block's run: steps that end a
row are filled by hand and their shared memory is copied into again two steps
later, for the next rows."""
import numpy as np
import pytest

import _tree as T
from test_gpu_logprob_range import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V,extra", [(8192 + 149, 0), (2 * 8192 - 3, 5), (8191, 1), (16384 + 1025, 3), (3 * 8192 + 2, 2)])
def test_logprobs_of_rows_that_end_inside_a_step(dtype, V, extra):
    """Rows rise or fall in turn, so that what a row's end left behind would show in the next one."""
    import torch
    R = 900
    g = torch.Generator(device="cuda").manual_seed(V)
    flat = torch.zeros(R * (V + extra) + 8, device="cuda")
    flat = flat if dtype == T.F32 else flat.bfloat16()
    x = torch.as_strided(flat, (R, V), (V + extra, 1), extra)
    ramp = torch.linspace(-3.0, 3.0, V, device="cuda")
    x.copy_(torch.randn((R, V), generator=g, device="cuda") * 0.1 + ramp * torch.where(torch.arange(R, device="cuda") % 2 == 0, 1.0, -1.0)[:, None])
    tokens = np.random.default_rng(V).integers(0, V, R).astype(np.int32)
    _check(x, tokens, 1.0, 6)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
def test_logprobs_of_rows_past_32_bits(dtype):
    """Rows more than 2^31 elements apart, from an odd address."""
    import torch
    V, ld = 9001, 2 ** 31 + 11
    flat = torch.empty(ld + V + 1, dtype=torch.float32 if dtype == T.F32 else torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (2, V), (ld, 1), 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn((2, V), generator=g, device="cuda"))
    _check(x, np.array([V - 1, 4], np.int32), 1.0, 5)
