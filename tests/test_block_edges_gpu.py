"""The operators around the layer at the ends of their ranges: rows whose squares leave fp32,
8-bit codes at their borders, scales whose product leaves fp32, and activations far from 0.
Bounds are derived as in test_block_gpu.py: a rounding is off by half a step."""

import pytest
import torch

import diffusion_transformer_moe_b200 as nm
from tests.test_block_gpu import (BF, E4M3, F32, clean, gen, randn)

pytestmark = pytest.mark.gpu


# ---- 8-bit rows ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(3, 8), (700, 1032), (2000, 512), (5, 16384)])
@pytest.mark.parametrize("size", [3.0, 1e-18, 1e-30, 1e-36, 1e-38, 1e30, 5e37])
def test_codes_are_those_of_the_quotient(T, d, dtype, size):
    # q = e4m3(x / scale): the code that the quotient in fp32 has, not a neighbour's
    x = randn(gen(T + d), T, d, dtype=F32, scale=size).to(dtype)
    x[0, 1], x[1, 2] = 0.0, -0.0
    q, scale = nm.quantize_rows(x)
    clean()
    assert torch.equal(q.view(torch.uint8),
                       (x.float() / scale[:, None]).to(E4M3).view(torch.uint8))
    # a norm's y in fp32 is what its q holds
    w = randn(gen(d), d, dtype=F32, scale=size)
    n = nm.rms_norm(randn(gen(T), T, d, dtype=F32), w, out="both")
    clean()
    assert torch.equal(n.q.view(torch.uint8),
                       (n.y / n.scale[:, None]).to(E4M3).view(torch.uint8))


def test_codes_of_rows_with_infinities():
    x = randn(gen(3), 4, 520)
    x[1, 5], x[2, 7], x[2, 9] = float("inf"), float("-inf"), float("nan")
    q, scale = nm.quantize_rows(x)
    clean()
    # finite / inf is 0 (of either sign), inf / inf and a row with a NaN are NaN
    got, want = q.float(), x.float() / scale[:, None]
    assert float(scale[1]) == float("inf") and bool(scale[2].isnan())
    assert torch.equal(got.isnan(), want.isnan())
    assert bool((got[1].nan_to_num(0) == 0).all()) and bool(got[3].isfinite().all())
