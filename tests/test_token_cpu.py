"""Refusals of the 4-bit products with scales per group and of the sampler: all before any HIP call, so no GPU is
needed.  What the binding hands over, and pins of their oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.token_oracle as T
import ternary_weight_quantized_q2_amd as q2
from tests.test_fused_binding_cpu import lib as recorder  # noqa: F401

FAKE = 1 << 20          # 256-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return q2.load()


def epi(activation=0, flags=0, bias=None, gate=None, residual=None):
    return ctypes.byref(q2.Epilogue(activation, flags, bias, gate, residual))


def test_matvec_argument_errors(lib):
    def L(x=FAKE, w=FAKE, s=FAKE, z=FAKE, g=64, fl=0, e=None, y=FAKE << 4, m=3, n=8, k=256):
        return lib.q4_matvec(x, w, s, z, g, fl, e, y, m, n, k, None)

    assert L(m=-1) == q2.Q2_ERR_ARG and L(n=-1) == q2.Q2_ERR_ARG and L(k=-32) == q2.Q2_ERR_ARG
    assert L(fl=2) == q2.Q2_ERR_ARG and b"flag" in lib.q2_last_error()
    for g in (0, -32, 16, 48, 96, 127, 160, 1 << 40, -2 ** 63, 2 ** 63 - 1):
        assert L(g=g) == q2.Q2_ERR_SHAPE, g
    assert L(g=512) == q2.Q2_ERR_SHAPE and b"multiple of the group" in lib.q2_last_error()
    assert L(k=(1 << 24) + 64) == q2.Q2_ERR_SHAPE and b"16777216" in lib.q2_last_error()
    assert L(m=1 << 50) == q2.Q2_ERR_ARG and L(n=1 << 50) == q2.Q2_ERR_ARG
    for name in ("x", "w", "s", "y"):
        assert L(**{name: None}) == q2.Q2_ERR_ARG, name
        assert L(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    assert L(x=FAKE + 8) == q2.Q2_ERR_ALIGN and L(w=FAKE + 8) == q2.Q2_ERR_ALIGN and L(z=FAKE + 1) == q2.Q2_ERR_ALIGN
    assert L(z=None, fl=q2.Q4_ZERO_CODES) == q2.Q2_ERR_ARG and b"zero points" in lib.q2_last_error()
    assert L(e=epi(activation=5)) == q2.Q2_ERR_ARG and L(e=epi(flags=8)) == q2.Q2_ERR_ARG
    assert L(e=epi(flags=q2.Q2_EPI_GATED), n=7) == q2.Q2_ERR_SHAPE
    assert L(e=epi(bias=FAKE + 2)) == q2.Q2_ERR_ALIGN and L(e=epi(residual=FAKE + 2)) == q2.Q2_ERR_ALIGN
    assert L(y=FAKE + 512) == q2.Q2_ERR_ARG and b"overlaps x" in lib.q2_last_error()
    # empty outputs touch nothing
    assert L(m=0, x=None, y=None) == q2.Q2_OK and L(n=0, w=None, s=None, z=None, y=None) == q2.Q2_OK


def test_sample_argument_errors(lib):
    def S(lg=FAKE, b=4, v=100, ld=100, fl=0, u=FAKE, t=FAKE, p=FAKE, ws=FAKE, wb=1 << 40, **c):
        s = q2.Sampling(1.0, 0, 1.0, 0.0, *(c.get(n) for n in ("tr", "kr", "pr", "mr")))
        return lib.q2_sample(lg, b, v, ld, fl, ctypes.addressof(s), u, t, p, ws, wb, None)

    assert S(b=-1) == q2.Q2_ERR_ARG and S(v=-1) == q2.Q2_ERR_ARG and S(fl=2) == q2.Q2_ERR_ARG
    assert S(v=0) == q2.Q2_ERR_SHAPE and S(v=(1 << 24) + 1, ld=1 << 25) == q2.Q2_ERR_SHAPE
    assert S(b=(1 << 30) + 1) == q2.Q2_ERR_SHAPE
    assert S(ld=99) == q2.Q2_ERR_ARG and S(ld=-1) == q2.Q2_ERR_ARG and S(ld=2 ** 63 - 1) == q2.Q2_ERR_ARG
    for name in ("lg", "u", "t", "p"):
        assert S(**{name: None}) == q2.Q2_ERR_ARG, name
        assert S(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    assert S(lg=FAKE + 2) == q2.Q2_ERR_ALIGN
    for name in ("tr", "kr", "pr", "mr"):
        assert S(**{name: FAKE + 2}) == q2.Q2_ERR_ALIGN, name
    assert S(b=0, lg=None, u=None, t=None, p=None) == q2.Q2_OK
    need = q2.sample_workspace_bytes(4, 100000)
    assert need > 0 and q2.sample_workspace_bytes(4, 100) == 0 and q2.sample_workspace_bytes(4, (1 << 24) + 1) == 0
    assert q2.sample_workspace_bytes(0, 100000) == 0 and q2.sample_workspace_bytes(-1, 100000) == 0
    assert q2.sample_workspace_bytes(2 ** 63 - 1, 2 ** 63 - 1) == 0 and q2.sample_workspace_bytes(-2 ** 63, 5) == 0
    big = dict(v=100000, ld=100000)
    assert S(wb=need - 1, **big) == q2.Q2_ERR_WORKSPACE and S(ws=None, **big) == q2.Q2_ERR_ARG
    assert S(ws=FAKE + 64, **big) == q2.Q2_ERR_ALIGN


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------

bf, u8, f16 = torch.bfloat16, torch.uint8, torch.float16


def test_binding_refuses_what_does_not_fit(recorder):  # noqa: F811
    x, w, s = torch.zeros((0, 128), dtype=bf), torch.zeros((0, 64), dtype=u8), torch.zeros((0, 2), dtype=f16)
    with pytest.raises(ValueError, match="packed4"):
        q2.q4_matvec(x, torch.zeros((0, 63), dtype=u8), s)
    with pytest.raises(ValueError, match="do not divide"):
        q2.q4_matvec(x, w, torch.zeros((0, 3), dtype=f16))
    with pytest.raises(ValueError, match="do not divide"):
        q2.q4_matvec(x, w, torch.zeros((0, 0), dtype=f16))
    with pytest.raises(ValueError, match="zero"):
        q2.q4_matvec(x, w, s, torch.zeros((0, 2), dtype=u8))
    with pytest.raises(ValueError, match="zero"):
        q2.q4_matvec(x, w, s, torch.zeros((0, 2)))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        q2.q2_sample(torch.zeros((0, 8), dtype=f16), torch.zeros(0))
    with pytest.raises(ValueError, match="u: expected"):
        q2.q2_sample(torch.zeros((0, 8)), torch.zeros(1))
    with pytest.raises(ValueError, match="top_k"):
        q2.q2_sample(torch.zeros((0, 8)), torch.zeros(0), top_k=torch.zeros(0))
    assert recorder.calls == []


def test_outputs_of_empty_inputs_are_on_the_device(recorder):  # noqa: F811
    q2.q4_matvec(torch.zeros((4, 0), dtype=bf), torch.zeros((6, 0), dtype=u8), torch.zeros((6, 0), dtype=f16))
    q2.q2_sample(torch.zeros((0, 8)), torch.zeros(0))
    assert recorder.calls == ["q4_matvec", "q2_sample"] and recorder.made == ["cuda:0"] * 3


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def test_weight_by_hand():
    # row 0: codes 1, 2, 3, 4, ... ; two groups of two inputs each
    packed = np.array([[0x21, 0x43], [0xF0, 0x8F]], np.uint8)
    scale = np.array([[1.0, 10.0], [0.5, -2.0]])
    assert T.weight(packed, scale, None).tolist() == [[-7.0, -6.0, -50.0, -40.0], [-4.0, 3.5, -14.0, 0.0]]
    assert T.weight(packed, scale, np.array([[0x31], [0x0F]], np.uint8)).tolist() == \
        [[0.0, 1.0, 0.0, 10.0], [-7.5, 0.0, -30.0, -16.0]]
    assert T.weight(packed, scale, np.array([[0.5, 1.0], [2.0, 15.5]])).tolist() == \
        [[0.5, 1.5, 20.0, 30.0], [-1.0, 6.5, 1.0, 15.0]]
    three = np.array([[0x10, 0x02]], np.uint8)              # zero points of three groups: 0, 1, 2
    assert T.weight(np.array([[0x55] * 3], np.uint8), np.ones((1, 3)), three).tolist() == [[5, 5, 4, 4, 3, 3]]


def test_sample_by_hand():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))              # order 1, 2, 0, 3 with p = 4, 2, 1, 1 of 8
    for u, t, p in ((0.0, 1, 0.5), (0.49, 1, 0.5), (0.51, 2, 0.25), (0.74, 2, 0.25), (0.76, 0, 0.125), (0.88, 3, 0.125),
                    (0.999, 3, 0.125), (1.0, 3, 0.125), (7.0, 3, 0.125), (-1.0, 1, 0.5), (math.nan, 1, 0.5)):
        got = T.sample_row(l, u)
        assert got[0] == t and abs(got[1] - p) < 1e-12, u
    assert T.sample_row(l, 0.9, top_k=2) == (2, pytest.approx(1 / 3))
    assert T.sample_row(l, 0.99, top_k=3) == (0, pytest.approx(1 / 7))     # of two equal ones the lower token stays
    assert T.sample_row(l, 0.99, top_p=0.74) == (2, pytest.approx(1 / 3)) and T.sample_row(l, 0.99, top_p=0.4) == (1, 1.0)
    assert T.sample_row(l, 0.99, min_p=0.3) == (2, pytest.approx(1 / 3)) and T.sample_row(l, 0.99, min_p=0.2)[0] == 3
    assert T.sample_row(l, 0.99, min_p=0.2, top_k=3, top_p=0.8) == (2, pytest.approx(1 / 3))   # 4, 2 of 7 reach 0.8
    assert T.sample_row(l, 0.79, temperature=0.5) == (2, pytest.approx(4 / 22))              # squares: 16, 4, 1, 1
    for off in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=math.nan), dict(top_k=1), dict(top_p=0.0),
                dict(min_p=1.5)):
        assert T.sample_row(l, 0.99, **off) == (1, 1.0)
    assert T.sample_row([0.0, 0.0], 0.99, min_p=1.0)[0] == 1 and T.sample_row([-math.inf, math.nan], 0.5) == (-1, 0.0)
    assert T.sample_row([math.inf, 0.0, math.inf], 0.6) == (2, 0.5)
    assert T.sample_row([math.inf, 0.0], 0.9, temperature=math.inf) == (0, 1.0)
