"""The residual norm's gradient and outputs at the ends of float32's range, and with a gamma that is not
finite, against the oracle (oracle.norm), GB300 only.

Tolerances as in test_gpu_norm.py: n three roundings of 2^-24 and half a step of its type; dx half a step,
eight roundings of each summand and width + 3 of the dot product's terms; dgamma tokens + 4.
"""

import numpy as np
import pytest

from oracle import norm
from helpers import to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mb():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mlp_block_backprop_gb300 as mb
    yield mb
    assert mb.mlpblk_last_error() == mb.MLPBLK_OK


def _t(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
def test_mean_squares_below_the_normal_range(mb, dtype, block):
    """eps = 0 and rows of 2^-65: their squares are 2^-130, exact, and rstd is 2^65."""
    import torch
    T, d = 5, 300
    rng = np.random.default_rng(3)
    x = rng.choice([-1.0, 1.0, 2.0], (T, d)) * 2.0 ** -np.arange(60, 70, 2)[:, None]
    x, gamma = _t(x, dtype), _t(rng.choice([0.5, 1.0, 1.5], d), dtype)
    op = mb.AddRmsNorm(T, d, 0.0, dtype, block)
    codes, n = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(x)
    scales = torch.empty(T, 3 if block else 1, device="cuda")
    op.forward(x, gamma, codes, scales, n=n)
    ref_n, ref_codes, ref_scales, ref_r = norm.forward(to_np(x), to_np(gamma), 0.0, block)
    np.testing.assert_allclose(to_np(op.rstd), ref_r, rtol=2.0 ** -23)
    np.testing.assert_allclose(to_np(n), ref_n, rtol=3 * U + (2.0 ** -8 if dtype == "bf16" else U))
    np.testing.assert_array_equal(to_np(scales), ref_scales.astype(np.float64))
    np.testing.assert_array_equal(to_np(codes), ref_codes)
