"""GPU tests of the 4-bit products with scales per group and of the sampler at the limits of what they take: zero points
and inputs of extreme sizes, outputs that are inputs, rows that workgroups share."""
import numpy as np
import pytest
import torch

import oracle.q2_oracle as O
import oracle.token_oracle as T
import ternary_weight_quantized_q2_amd as q2
from tests.test_fused_gpu import check_terms
from tests.test_parity_gpu import DEV, acts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU parity tests need a GPU; they must not be skipped silently"
    torch.cuda.set_device(0)
    q2.load()
    yield


SMALL_ZEROS = [2.0 ** -24, -2.0 ** -24, 2.0 ** -20, -2.0 ** -17, 1.5 * 2.0 ** -14, 1025 * 2.0 ** -20, -1.25]


def small_zero_weights(seed, n, k, group):
    """Three of four columns have codes of 0 alone and zero points that are no code, so that nothing but the zero points
    is left; the others' codes are any."""
    g = np.random.default_rng([seed, n, k])
    packed = g.integers(0, 256, (n, k // 2)).astype(np.uint8)
    packed[np.arange(n) % 4 != 3] = 0
    scale = (g.random((n, k // group)) + 0.5).astype(np.float16)
    zero = np.repeat(np.resize(SMALL_ZEROS, n)[:, None], k // group, axis=1).astype(np.float16)
    zero[5::9] = g.choice(SMALL_ZEROS, zero[5::9].shape)
    return packed, scale, zero


@pytest.mark.parametrize("group,k", [(32, 64), (64, 192), (128, 128), (32, 1120), (64, 2560), (128, 1280), (256, 2560)])
@pytest.mark.parametrize("m", [1, 4, 7, 20, 40])
def test_small_zero_points(group, k, m):
    """Every output by its own terms, x z s.  A sum of x over up to 128 inputs is off by at most 128 2^-24 sum |x|, 8.7e-5
    of the root of the sum of the terms' squares; the sum over K / 32 groups or less by 2^-24 of at most sqrt(K) times that
    root each, 2.5e-4; and the bar is 1e-3."""
    packed, scale, zero = small_zero_weights(501, 50, k, group)
    xb, x = acts(501, m, k)
    y = q2.q4_matvec(x, *(torch.from_numpy(t).to(DEV) for t in (packed, scale, zero)))
    check_terms(y, O.bf16_to_f64(xb), T.weight(packed, scale, zero))


@pytest.mark.parametrize("m,n", [(33, 20010), (64, 96016)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_small_zero_points_of_wide_weights(group, m, n):
    """The same with 32 and 64 rows per decoded weight; sampled columns."""
    packed, scale, zero = small_zero_weights(502, n, 384, group)
    cols = np.unique(np.concatenate([np.arange(40), n - 1 - np.arange(40), np.random.default_rng(502).choice(n, 100)]))
    xb, x = acts(502, m, 384)
    y = q2.q4_matvec(x, *(torch.from_numpy(t).to(DEV) for t in (packed, scale, zero)))
    check_terms(y[:, torch.from_numpy(cols).to(DEV)], O.bf16_to_f64(xb), T.weight(packed[cols], scale[cols], zero[cols]))
