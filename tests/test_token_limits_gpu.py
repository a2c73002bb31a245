"""GPU tests of the 4-bit products with scales per group and of the sampler at the limits of what they take: zero points
and inputs of extreme sizes, outputs that are inputs, rows that workgroups share."""
import numpy as np
import pytest
import torch

import oracle.q2_oracle as O
import oracle.token_oracle as T
import ternary_weight_quantized_q2_amd as q2
from tests.test_fused_gpu import check_terms, rnd
from tests.test_parity_gpu import DEV, acts
from tests.test_token_gpu import uniform

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


def largest_inputs(m, k):
    """bf16 rows whose sum of |x| over any 128 inputs is 0.99 2^126, as bits and on the device."""
    g = np.random.default_rng([503, m, k])
    xb = np.where(g.random((m, k)) < 0.9, 0x7AFD, 0xFAFD).astype(np.uint16)    # +-(1 + 125 / 128) 2^118
    return xb, torch.from_numpy(xb.view(np.int16)).to(DEV).view(torch.bfloat16)


@pytest.mark.parametrize("group,k", [(32, 96), (64, 64), (128, 128), (64, 1280), (128, 2560), (512, 1024), (1280, 2560)])
@pytest.mark.parametrize("zero", [None, 15.0, 16.0])
@pytest.mark.parametrize("m", [1, 9, 40])
def test_largest_inputs(group, k, zero, m):
    """The largest x that are promised to work."""
    g = np.random.default_rng(504)
    packed = g.integers(0, 256, (30, k // 2)).astype(np.uint8)
    scale = ((g.random((30, k // group)) + 0.5) * 2.0 ** -12).astype(np.float16)
    z = None if zero is None else np.full(scale.shape, zero, np.float16)
    xb, x = largest_inputs(m, k)
    y = q2.q4_matvec(x, *(None if t is None else torch.from_numpy(t).to(DEV) for t in (packed, scale, z)))
    check_terms(y, O.bf16_to_f64(xb), T.weight(packed, scale, z))


def test_largest_inputs_of_more_rows_than_the_grid():
    """The same in one group of 512 inputs, whose sum of |x| is beyond fp32, for more rows than the grid's second
    dimension takes."""
    m, k = 65535 * 64 + 70, 512
    g = np.random.default_rng(505)
    packed = g.integers(0, 256, (2, k // 2)).astype(np.uint8)
    scale = np.full((2, 1), 2.0 ** -12, np.float16)
    xb, x = largest_inputs(50, k)
    x = torch.abs(x).repeat(m // 50 + 1, 1)[:m].contiguous()
    y = q2.q4_matvec(x, torch.from_numpy(packed).to(DEV), torch.from_numpy(scale).to(DEV))
    check_terms(y[:50], O.bf16_to_f64(xb & 0x7FFF), T.weight(packed, scale, None))
    whole = y[:m // 50 * 50].view(-1, 50, 2)
    assert (whole == whole[0]).all() and torch.equal(y[m // 50 * 50:], y[:m % 50])


@pytest.mark.parametrize("b,v", [(1, 300), (300, 300), (3, 50021), (100, 60000)])
@pytest.mark.parametrize("settings", [dict(), dict(top_k=40, top_p=0.9), dict(temperature=0.0), dict(temperature=2.0, top_k=3000)])
def test_random_numbers_in_an_output(b, v, settings):
    """prob may be u, and token the memory of u."""
    logits, u = (rnd(b, b, v) * 3).to(DEV), uniform(b, b).to(DEV)
    want = q2.q2_sample(logits, u, **settings)
    own = u.clone()
    got = q2.q2_sample(logits, own, prob=own, **settings)
    assert got.prob is own and all(torch.equal(a, c) for a, c in zip(got, want))
    own = u.clone()
    got = q2.q2_sample(logits, own, token=own.view(torch.int32), **settings)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    wide = torch.cat([u, u])
    if b > 1:
        with pytest.raises(q2.Q2Error, match="overlaps u"):
            q2.q2_sample(logits, wide[:b], prob=wide[1:b + 1], **settings)
    with pytest.raises(q2.Q2Error, match="overlaps the logits"):
        q2.q2_sample(logits, u, prob=logits.view(-1)[-b:], **settings)


def test_outputs_beside_the_logits():
    """Outputs in the columns that rows of logits have behind them."""
    wide = (rnd(5, 6, 320) * 3).to(DEV)
    want = q2.q2_sample(wide[:, :300], uniform(5, 6).to(DEV), top_p=0.9)
    token, prob = wide[2, 300:306].view(torch.int32), wide[4, 310:316]
    got = q2.q2_sample(wide[:, :300], uniform(5, 6).to(DEV), top_p=0.9, token=token, prob=prob)
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and got.prob is prob
