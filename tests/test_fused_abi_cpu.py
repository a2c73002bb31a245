"""Refusals of the fused and grouped linears, the router and the combination: all
before any HIP call, so no GPU is needed.  Then pins of their oracle."""
import ctypes
import math

import numpy as np
import pytest

import oracle.fused_oracle as F
import ternary_weight_quantized_q2_amd as q2

FAKE = 1 << 20          # 256-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return q2.load()


def epi(activation=0, flags=0, bias=None, gate=None, residual=None):
    return ctypes.byref(q2.Epilogue(activation, flags, bias, gate, residual))


def test_fused_argument_errors(lib):
    need = lib.q2_linear_fused_workspace_bytes(16, 8, 128, 8)
    assert need >= lib.q2_lowrank_workspace_bytes(16, 8)

    def L(x=FAKE, w=FAKE, s=FAKE, A=FAKE, B=FAKE, r=0, e=None, y=FAKE, m=16, n=8, k=128, ws=FAKE, wb=1 << 30):
        return lib.q2_linear_fused(x, w, s, A, B, r, e, y, m, n, k, ws, wb, None)

    assert L(m=-1) == q2.Q2_ERR_ARG and L(n=-1) == q2.Q2_ERR_ARG
    assert L(k=100) == q2.Q2_ERR_SHAPE and L(k=(1 << 24) + 128) == q2.Q2_ERR_SHAPE
    assert L(r=-1) == q2.Q2_ERR_ARG and L(r=65536) == q2.Q2_ERR_ARG
    for name in ("x", "w", "s", "y"):
        assert L(**{name: None}) == q2.Q2_ERR_ARG, name
        assert L(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    assert L(x=FAKE + 8) == q2.Q2_ERR_ALIGN and L(w=FAKE + 8) == q2.Q2_ERR_ALIGN
    assert L(r=8, A=None) == q2.Q2_ERR_ARG and L(r=8, B=FAKE + 1) == q2.Q2_ERR_ALIGN
    assert L(r=8, A=FAKE + 2) == q2.Q2_ERR_ALIGN
    assert L(r=8, wb=need - 1) == q2.Q2_ERR_WORKSPACE
    assert L(r=8, ws=None) == q2.Q2_ERR_ARG and L(r=8, ws=FAKE + 16) == q2.Q2_ERR_ALIGN
    assert L(e=epi(activation=5)) == q2.Q2_ERR_ARG and L(e=epi(flags=8)) == q2.Q2_ERR_ARG
    assert L(e=epi(flags=q2.Q2_EPI_GATED), n=7) == q2.Q2_ERR_SHAPE and b"halves" in lib.q2_last_error()
    assert L(e=epi(bias=FAKE + 2)) == q2.Q2_ERR_ALIGN and L(e=epi(gate=FAKE + 1)) == q2.Q2_ERR_ALIGN
    assert L(e=epi(residual=FAKE + 2)) == q2.Q2_ERR_ALIGN
    assert L(e=epi(flags=q2.Q2_EPI_OUT_BF16), y=FAKE + 1) == q2.Q2_ERR_ALIGN
    # empty outputs touch nothing
    assert L(m=0, x=None, y=None) == q2.Q2_OK and L(n=0, w=None, s=None, y=None) == q2.Q2_OK
    assert lib.q4_linear_fused(FAKE, FAKE, FAKE, None, None, FAKE, 3, 5, 128, None) == q2.Q2_ERR_ARG
    assert lib.q4_linear_fused(FAKE, FAKE, FAKE, FAKE, epi(activation=9), FAKE, 3, 5, 128, None) == q2.Q2_ERR_ARG
    assert lib.q4_linear_fused(FAKE, FAKE, FAKE, FAKE + 1, None, FAKE, 3, 5, 128, None) == q2.Q2_ERR_ALIGN
    assert lib.q4_linear_fused(None, FAKE, FAKE, FAKE, None, None, 0, 5, 128, None) == q2.Q2_OK


def test_grouped_argument_errors(lib):
    def G(x=FAKE, xr=10, idx=FAKE, off=FAKE, w=FAKE, s=FAKE, e=None, y=FAKE, r=20, E=4, n=8, k=128, ws=FAKE, wb=1 << 40):
        return lib.q2_linear_grouped(x, xr, idx, off, w, s, e, y, r, E, n, k, ws, wb, None)

    assert G(r=-1) == q2.Q2_ERR_ARG and G(E=-1) == q2.Q2_ERR_ARG and G(xr=-1) == q2.Q2_ERR_ARG
    assert G(k=64) == q2.Q2_ERR_SHAPE and G(E=65537) == q2.Q2_ERR_SHAPE
    assert G(r=1 << 31) == q2.Q2_ERR_SHAPE and G(xr=1 << 31) == q2.Q2_ERR_SHAPE
    assert G(idx=None) == q2.Q2_ERR_ARG and b"x_rows" in lib.q2_last_error()
    assert G(idx=None, xr=20, off=None) == q2.Q2_ERR_ARG
    assert G(idx=FAKE + 2) == q2.Q2_ERR_ALIGN and G(off=FAKE + 2) == q2.Q2_ERR_ALIGN
    for name in ("x", "w", "s", "y"):
        assert G(**{name: None}) == q2.Q2_ERR_ARG, name
        assert G(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    assert G(e=epi(gate=FAKE)) == q2.Q2_ERR_ARG and G(e=epi(residual=FAKE)) == q2.Q2_ERR_ARG
    assert G(e=epi(flags=q2.Q2_EPI_GATED), n=9) == q2.Q2_ERR_SHAPE
    need = lib.q2_linear_grouped_workspace_bytes(5000, 4, 4096, 2048)
    if need:
        assert G(r=5000, n=4096, k=2048, wb=need - 1) == q2.Q2_ERR_WORKSPACE
        assert G(r=5000, n=4096, k=2048, ws=None) == q2.Q2_ERR_ARG
        assert G(r=5000, n=4096, k=2048, ws=FAKE + 64) == q2.Q2_ERR_ALIGN
    for empty in (dict(r=0), dict(E=0), dict(n=0)):
        assert G(x=None, off=None, w=None, s=None, y=None, **empty) == q2.Q2_OK
    assert lib.q4_linear_grouped(FAKE, 10, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, 20, 4, 8, 128,
                                 None) == q2.Q2_ERR_ARG


def test_route_and_combine_argument_errors(lib):
    def R(lg=FAKE, t=100, e=8, k=2, fl=0, ex=FAKE, wt=FAKE, off=FAKE, tok=FAKE, sl=FAKE, ws=FAKE, wb=1 << 30):
        return lib.q2_route(lg, t, e, k, fl, ex, wt, off, tok, sl, ws, wb, None)

    assert R(t=-1) == q2.Q2_ERR_ARG and R(fl=4) == q2.Q2_ERR_ARG
    assert R(k=0) == q2.Q2_ERR_SHAPE and R(k=9) == q2.Q2_ERR_SHAPE and R(e=0) == q2.Q2_ERR_SHAPE
    assert R(e=1025) == q2.Q2_ERR_SHAPE and R(e=100, k=65) == q2.Q2_ERR_SHAPE
    assert R(t=1 << 30, k=2) == q2.Q2_ERR_SHAPE
    for name in ("lg", "ex", "wt", "off", "tok", "sl"):
        assert R(**{name: None}) == q2.Q2_ERR_ARG, name
        assert R(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    need = lib.q2_route_workspace_bytes(100, 8, 2)
    assert need > 0 and lib.q2_route_workspace_bytes(64, 8, 2) == 0 and lib.q2_route_workspace_bytes(100, 8, 9) == 0
    assert R(wb=need - 1) == q2.Q2_ERR_WORKSPACE and R(ws=None) == q2.Q2_ERR_ARG and R(ws=FAKE + 4) == q2.Q2_ERR_ALIGN

    def C(z=FAKE, r=10, sl=FAKE, wt=FAKE, res=None, y=FAKE, t=4, k=2, n=8, fl=0):
        return lib.q2_combine(z, r, sl, wt, res, y, t, k, n, fl, None)

    assert C(t=-1) == q2.Q2_ERR_ARG and C(fl=8) == q2.Q2_ERR_ARG
    assert C(k=65) == q2.Q2_ERR_SHAPE and C(r=1 << 31) == q2.Q2_ERR_SHAPE and C(n=1 << 47) == q2.Q2_ERR_SHAPE
    for name in ("z", "sl", "wt", "y"):
        assert C(**{name: None}) == q2.Q2_ERR_ARG, name
        assert C(**{name: FAKE + 1}) == q2.Q2_ERR_ALIGN, name
    assert C(res=FAKE + 2) == q2.Q2_ERR_ALIGN and C(res=FAKE + 1, fl=4) == q2.Q2_ERR_ALIGN
    assert C(z=None, sl=None, wt=None, y=None, t=0) == q2.Q2_OK
    assert C(z=None, sl=None, wt=None, y=None, n=0) == q2.Q2_OK


def test_workspace_sizes_at_the_limits(lib):
    big, small = 2 ** 63 - 1, -2 ** 63
    f, g = lib.q2_linear_fused_workspace_bytes, lib.q2_linear_grouped_workspace_bytes
    assert f(0, 8, 128, 4) == 0 and f(small, 8, 128, 4) == 0 and f(4, 8, 128, -1) == 0 and f(4, 8, 128, 65536) == 0
    assert f(big, big, big, 0) == 0 and g(big, 4, 8, 128) == 0 and g(4, big, 8, 128) == 0 and g(4, 0, 8, 128) == 0
    assert lib.q2_route_workspace_bytes(big, 8, 2) == 0 and lib.q2_route_workspace_bytes(small, 8, 2) == 0


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def test_activation_values():
    # erf(1 / sqrt 2) = 0.682689492137086 (the one-sigma probability), tanh and exp from closed forms
    assert F.activate("gelu", np.array([1.0]))[0] == pytest.approx(0.841344746068543, abs=1e-15)
    assert F.activate("silu", np.array([math.log(3.0)]))[0] == pytest.approx(0.75 * math.log(3.0), abs=1e-15)
    v = np.linspace(-6, 6, 101)
    assert np.abs(F.activate("gelu", v) - F.activate("gelu_tanh", v)).max() < 5e-4
    for name in ("gelu", "gelu_tanh", "silu"):
        assert np.allclose(F.activate(name, v) - F.activate(name, -v), v)      # x P(x) + x P(-x) = x
        assert F.activate(name, np.array([-1000.0]))[0] == pytest.approx(0.0)
    assert F.activate("relu", np.array([-2.0, 3.0])).tolist() == [0.0, 3.0]


def test_slopes_bound_the_activations():
    v = np.linspace(-8, 8, 200001)
    for name, s in F.SLOPE.items():
        d = np.abs(np.diff(F.activate(name, v)) / np.diff(v)).max()
        assert s * 0.995 <= d * 1.001 and d <= s


def test_epilogue_by_hand():
    z = np.array([[1.0, -2.0, 3.0, 4.0]])
    assert F.epilogue(z, "relu", bias=[1, 1, 1, 1]).tolist() == [[2, 0, 4, 5]]
    assert F.epilogue(z, "relu", True, bias=[0, 3, 1, 0]).tolist() == [[4.0, 4.0]]     # relu(1)*4, relu(1)*4
    assert F.epilogue(z, "none", True, gate=[2, 3], residual=[[10, 20]]).tolist() == [[16.0, -4.0]]


def test_grouped_products_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 5.0]])
    w = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[1.0, 1.0]]])
    z = F.grouped_products(x, w, [0, 1, 1, 3], [1, 0, 7])
    assert z.tolist() == [[3.0], [3.0], [0.0]]
    assert np.isnan(F.grouped_products(x, w, [1, 2, 2, 2])[0, 0])


def test_route_by_hand():
    ln = math.log
    logits = np.array([[ln(1), ln(3), ln(3), ln(1)], [-math.inf, ln(2), math.nan, -math.inf]])
    ex, w, off, tok, slot = F.route(logits, 2, False)
    assert ex.tolist() == [[1, 2], [1, -1]] and w[0].tolist() == pytest.approx([3 / 8, 3 / 8]) and w[1].tolist() == [1, 0]
    assert off.tolist() == [0, 0, 2, 3, 3] and tok.tolist() == [0, 1, 0, -1] and slot.tolist() == [[0, 2], [1, -1]]
    assert F.route(logits, 2, True)[1][0].tolist() == pytest.approx([0.5, 0.5])
    assert F.route(np.array([[math.inf, 0.0, math.inf]]), 3, False)[1].tolist() == [[0.5, 0.5, 0.0]]


def test_combine_by_hand():
    z = np.array([[1.0], [10.0]])
    y = F.combine(z, np.array([[0, 1], [-1, 1], [2, -5]]), np.array([[2.0, 3.0]] * 3), np.array([[0.5]] * 3))
    assert y.tolist() == [[32.5], [30.5], [0.5]]


def test_route_workgroups_hold_few_enough_tokens_for_their_counts(lib):
    """A workgroup counts its tokens per expert in 16 bits: it must not have more than 65535 (k = E chooses every
    expert for each of them).  1024 experts: 2048 bytes of counts per workgroup."""
    for t in (65, 70001, 1023 * 65536, 1023 * 65536 + 1, 2 ** 26 - 1, 2 ** 26):
        groups = lib.q2_route_workspace_bytes(t, 1024, 1) // 2048
        assert groups * 65535 >= t, t


def test_workspace_queries_leave_the_message(lib):
    """A query is no failed call, whatever its sizes."""
    f, g = lib.q2_linear_fused_workspace_bytes, lib.q2_linear_grouped_workspace_bytes
    assert lib.q2_linear(None, None, None, None, -1, 1, 128, None) == q2.Q2_ERR_ARG
    detail = lib.q2_last_error()
    assert b"negative" in detail
    for k in (100, (1 << 24) + 128, -128):
        assert f(4, 8, k, 0) == 0 and f(4096, 8192, k, 0) == 0 and g(4096, 4, 8192, k) == 0
    assert f(1 << 40, 1 << 20, 128, 0) == 0 and f(4, 1 << 46, 128, 0) == 0 and g(1 << 20, 1 << 16, 1 << 30, 1 << 20) == 0
    assert lib.q2_last_error() == detail


def test_shape_errors_say_what_is_wrong(lib):
    """A refused size that is no K is not reported as one."""
    assert lib.q2_route(FAKE, 4, 1025, 2, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == q2.Q2_ERR_SHAPE
    assert lib.q2_linear_fused(FAKE, FAKE, FAKE, None, None, 0, epi(flags=q2.Q2_EPI_GATED), FAKE, 4, 7, 128, None, 0,
                               None) == q2.Q2_ERR_SHAPE
    name = lib.q2_strerror(q2.Q2_ERR_SHAPE)
    assert name.startswith(b"Q2_ERR_SHAPE") and b"128" not in name and b"halves" in lib.q2_last_error()


def test_outputs_that_overlap_what_others_read_are_refused(lib):
    """y over x, a residual that starts elsewhere in y or has another type, z."""
    m = n = k = 128
    far = FAKE + (1 << 20)

    def L(x=FAKE, y=far, **kw):
        return lib.q2_linear_fused(x, far << 4, far << 4, None, None, 0, epi(**kw), y, m, n, k, None, 0, None)

    bf = q2.Q2_EPI_OUT_BF16
    for y in (FAKE, FAKE + 2 * m * k - 4, FAKE - 4 * m * n + 4):
        assert L(y=y) == q2.Q2_ERR_ARG and b"overlaps x" in lib.q2_last_error()
    assert L(y=FAKE, residual=FAKE, flags=bf | q2.Q2_EPI_RESIDUAL_BF16) == q2.Q2_ERR_ARG      # x itself updated in place
    for res, flags in ((far + 4, 0), (far - 4, 0), (far, q2.Q2_EPI_RESIDUAL_BF16), (far, bf)):
        assert L(residual=res, flags=flags) == q2.Q2_ERR_ARG and b"residual" in lib.q2_last_error()
    assert lib.q4_linear_fused(FAKE, far, far, far, None, FAKE, m, n, k, None) == q2.Q2_ERR_ARG
    assert lib.q2_linear_grouped(FAKE, m, None, far, far, far, None, FAKE + 256, m, 1, n, k, None, 0, None) == q2.Q2_ERR_ARG
    assert lib.q4_linear_grouped(FAKE, m, None, far, far, far, far, None, FAKE, m, 1, n, k, None) == q2.Q2_ERR_ARG

    def C(y, res=None, fl=0):
        return lib.q2_combine(FAKE, 64, far << 2, far << 2, res, y, 16, 2, 64, fl, None)

    assert C(FAKE) == q2.Q2_ERR_ARG and C(FAKE + 4 * 64 * 64 - 4) == q2.Q2_ERR_ARG and b"overlaps z" in lib.q2_last_error()
    assert C(far, far + 8) == q2.Q2_ERR_ARG and C(far, far, q2.Q2_COMBINE_OUT_BF16) == q2.Q2_ERR_ARG
