"""Sizes whose launches would take 2^32 threads or more: refused by the plain linears and the rank-r branch (such a launch
runs in part and returns without an error), with y left as it was; the largest sizes below are computed."""
import numpy as np
import pytest
import torch

import oracle.q2_oracle as O
import ternary_weight_quantized_q2_amd as q2
from ternary_weight_quantized_q2_amd import inputs as I
from tests.test_parity_gpu import DEV, assert_close, dev_bits, q2_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU parity tests need a GPU; they must not be skipped silently"
    torch.cuda.set_device(0)
    q2.load()
    yield
    torch.cuda.empty_cache()


def empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def refused(call, y):
    y.fill_(7.0)
    with pytest.raises(q2.Q2Error) as e:
        call(y)
    assert e.value.status == q2.Q2_ERR_HIP
    assert all((part == 7).all() for part in y.view(-1).split(1 << 28))
    assert torch.ones(3, device=DEV).sum().item() == 3           # the device is as usable as before


def test_most_weight_rows():
    n, k = 2 ** 28, 128
    x = torch.ones((1, k), device=DEV, dtype=torch.bfloat16)
    p, s = empty(n, k // 4, dtype=torch.uint8), torch.ones((n, 1), device=DEV, dtype=torch.float16)
    p.fill_(0xAA)                                                # codes 2
    refused(lambda y: q2.q2_linear(x, p, s, y=y), empty(1, n, dtype=torch.float32))
    m = n - 16
    y = q2.q2_linear(x, p[:m], s[:m], y=torch.zeros((1, m), device=DEV))
    assert (y == k).all()


def test_most_rows_of_8_bit_activations():
    m, k, n = 2 ** 24, 128, 16
    p, s, p_ref, s_ref = q2_weights(371, n, k)
    xb = I.activations_bf16(371, 64, k)
    x = dev_bits(xb, torch.bfloat16).repeat(m // 64, 1)
    refused(lambda y: q2.q2_linear_a8(x, p, s, y=y), empty(m, n, dtype=torch.float32))
    y = q2.q2_linear_a8(x[:m - 1], p, s)
    assert_close(y[:64].cpu().numpy(), O.q2_linear_a8(xb, p_ref, s_ref))
    assert torch.equal(y[-63:], y[:63])


def test_most_rows_of_a_branch():
    m, k, n, r = 2 ** 26, 128, 8, 1
    p, s, p_ref, s_ref = q2_weights(372, n, k)
    ab, bb = I.lowrank_factors(372, r, k, n)
    A, B = dev_bits(ab, torch.float16), dev_bits(bb, torch.float16)
    xb = I.activations_bf16(372, 64, k)
    x = dev_bits(xb, torch.bfloat16).repeat(m // 64, 1)
    y = empty(m, n, dtype=torch.float32)
    refused(lambda y: q2.q2_linear_lowrank(x, p, s, A, B, y=y), y)
    refused(lambda y: q2.q2_linear_fused(x, p, s, A, B, y=y), y)
    for call in (q2.q2_linear_lowrank, q2.q2_linear_fused):
        got = call(x[:m - 16], p, s, A, B, y=y[:m - 16])
        assert_close(got[:64].cpu().numpy(), O.q2_linear_lowrank(xb, p_ref, s_ref, ab, bb))
        assert torch.equal(got[-16:], got[32:48])
        got.fill_(7.0)
