"""GPU tests of the fused and grouped linears against the float64 oracle.

Tolerance of an output: the product z is held to the linears' bar, |err z| <=
1e-3 of the RMS of z's row; the epilogue passes that on through the activation
(its largest slope) and the gate; the output type adds half a step of itself
(finfo.eps / 2 relative).  The epilogue's own fp32 arithmetic is a few ulps of
its terms, 2^-20 of them is allowed.
"""
import math

import numpy as np
import pytest
import scipy.special
import torch

import oracle.fused_oracle as F
import oracle.q2_oracle as O
import ternary_weight_quantized_q2_amd as q2
from ternary_weight_quantized_q2_amd import inputs as I
from tests.test_parity_gpu import DEV, acts, dev_bits, dev_u8, q2_weights

pytestmark = pytest.mark.gpu

ACTS = list(q2.ACTIVATIONS)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU parity tests need a GPU; they must not be skipped silently"
    torch.cuda.set_device(0)
    q2.load()
    yield


def q4_weights(cfg, n, k):
    p, s, z = I.q4_weights(cfg, n, k)
    return (dev_u8(p), dev_bits(s, torch.float16), dev_bits(z, torch.float16)), (p, s, z)


def weights(fmt, cfg, n, k):
    """(device arguments, float64 weight) of a seeded weight."""
    if fmt == "q2":
        p, s, p_ref, s_ref = q2_weights(cfg, n, k)
        return (p, s), O.unpack_q2(p_ref, s_ref).astype(np.float64)
    dev, ref = q4_weights(cfg, n, k)
    return dev, O.unpack_q4(*ref).astype(np.float64)


def fused(fmt):
    return q2.q2_linear_fused if fmt == "q2" else q2.q4_linear_fused


def grouped(fmt):
    return q2.q2_linear_grouped if fmt == "q2" else q2.q4_linear_grouped


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def host(t):
    return None if t is None else t.detach().cpu().double().numpy()


def tolerance(z, act, gated, bias, gate, residual, out_dtype):
    """Per-element bound on |y - oracle| (see the module's comment)."""
    v = z + (0 if bias is None else bias)
    dz = 1e-3 * np.sqrt(np.mean(z * z, axis=1, keepdims=True)) + 2.0 ** -20 * np.abs(v)
    slope = F.SLOPE[act]
    if gated:
        n = z.shape[1] // 2
        a, u = F.activate(act, v[:, :n]), v[:, n:]
        a_err = slope * dz[:, :n] + 2.0 ** -20 * np.abs(a)
        err = a_err * np.abs(u) + (np.abs(a) + a_err) * dz[:, n:]
        y = a * u
    else:
        y = F.activate(act, v)
        err = slope * dz + 2.0 ** -20 * np.abs(v)
    if gate is not None:
        y, err = y * gate, err * np.abs(gate)
    err = err + 2.0 ** -20 * np.abs(y)
    if residual is not None:
        y = y + residual
        err = err + 2.0 ** -20 * np.abs(residual)
    # half a step of the output type: relative to the value, and below the smallest normal number, where the steps
    # stop shrinking, half of the last step (smallest_normal * eps is the distance of neighbours there)
    t = torch.finfo(out_dtype)
    return y, err + (np.abs(y) + err) * t.eps / 2 + t.smallest_normal * t.eps / 2


def check(got, z, act="none", gated=False, bias=None, gate=None, residual=None, what=""):
    ref = F.epilogue(z, act, gated, host(bias), host(gate), host(residual))
    y, tol = tolerance(z, act, gated, host(bias), host(gate), host(residual), got.dtype)
    assert np.allclose(y, ref, rtol=1e-12, atol=1e-12)
    g = host(got)
    assert np.isfinite(g).all(), what
    bad = np.abs(g - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
                          f"{g[bad][0]} for {ref[bad][0]} +- {tol[bad][0]}"


# rows: one token, the GEMV's limit and beyond, tile edges; columns: not a multiple of anything, tile edges
SIZES = [(1, 64, 128), (1, 1000, 2560), (3, 37, 384), (16, 400, 1280), (17, 130, 640), (33, 1, 128), (64, 256, 512),
         (100, 513, 1152), (130, 200, 384), (257, 770, 1024), (300, 640, 1536), (1, 200, 12416), (16, 96, 12416),
         (9, 4200, 4224), (2, 9000, 640), (30, 70, 12416)]


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_plain_sizes(fmt, m, n, k):
    dev, w = weights(fmt, 301, n, k)
    xb, x = acts(301, m, k)
    z = O.bf16_to_f64(xb) @ w.T
    y = fused(fmt)(x, *dev)
    assert y.dtype == torch.float32
    check(y, z, what=f"{fmt} {m} {n} {k}")
    yb = fused(fmt)(x, *dev, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16)), "the bf16 output is not the f32 one rounded once"


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("m,n,k", [(8192, 1, 512), (4500, 1, 640), (8200, 3, 640), (5000, 9, 1152)])
def test_narrow_weights_over_many_rows(fmt, m, n, k):
    """Weights smaller than what the kernel prefetches."""
    dev, w = weights(fmt, 302, n, k)
    xb, x = acts(302, m, k)
    check_terms(fused(fmt)(x, *dev), O.bf16_to_f64(xb), w)


def check_terms(got, x, w):
    """got against x W^T, every element by the RMS sum of its own terms: a row's RMS over one to nine outputs may be
    far below the sums' rounding, and outputs of one row may differ in size by any factor."""
    bad = np.abs(host(got) - x @ w.T) > 1e-3 * np.sqrt((x * x) @ (w * w).T)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}"


# The kernel for many rows needs many tiles: wide weights, sampled columns (both factors' of a gated layer).
MANY = [(1531, 8120, 640, 40, False), (1531, 8120, 512, 0, True),
        (300, 32770, 512, 0, False), (1025, 9000, 1152, 0, True), (2000, 5250, 4224, 0, False), (700, 16400, 640, 5, True),
        (1500, 7000, 12416, 32, False), (1300, 8200, 2560, 64, True), (900, 12300, 512, 100, False)]


def sample(n, gated, seed):
    """Sorted sample of the output columns, the first and last ones in it, and of the weight rows behind them."""
    n_out = n // 2 if gated else n
    rng = np.random.default_rng(seed)
    cols = np.unique(np.concatenate([np.arange(40), n_out - 1 - np.arange(40), rng.choice(n_out, 60)]))
    return cols, np.concatenate([cols, cols + n_out]) if gated else cols


def spread_rows(seed, x):
    """bf16 bits whose rows have scales of their own, from 2^-60 to 2^60, one of them zero."""
    e = np.random.default_rng(seed).integers(-60, 61, (len(x), 1))
    e[len(x) // 3] = -1000
    return I.f32_to_bf16_bits(np.ldexp(O.bf16_to_f64(x), e).astype(np.float32))


@pytest.mark.parametrize("m,n,k,r,gated", MANY)
def test_many_rows(m, n, k, r, gated):
    codes = np.random.default_rng(315).integers(0, 3, (n, k)).astype(np.uint8)
    scales = I.q2_scales(315, n, k)
    p, s = q2.q2_pack(dev_u8(codes), torch.from_numpy(scales).to(DEV))
    cols, rows = sample(n, gated, 315)
    w = (codes[rows].astype(np.float64) - 1) * np.repeat(scales[rows].astype(np.float64), 128, axis=1)
    xb = spread_rows(315, I.activations_bf16(315, m, k))
    x = dev_bits(xb, torch.bfloat16)
    xd = O.bf16_to_f64(xb)
    z = xd @ w.T
    A = B = None
    if r:
        a, b = I.lowrank_factors(315, r, k, n, std=0.05)
        A, B = dev_bits(a, torch.float16), dev_bits(b, torch.float16)
        z = z + (xd @ O.f16_to_f64(a).T) @ O.f16_to_f64(b[rows]).T
    act = "relu" if gated else "none"                      # rows far from 1: what scales with them
    y = q2.q2_linear_fused(x, p, s, A, B, activation=act, gated=gated)
    sel = torch.from_numpy(cols).to(DEV)
    check(y[:, sel], z, act, gated, what="f32")
    assert (y[m // 3] == 0).all()
    yb = q2.q2_linear_fused(x, p, s, A, B, activation=act, gated=gated, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))
    # the epilogue, with ordinary rows
    xb = I.activations_bf16(316, m, k)
    x, xd = dev_bits(xb, torch.bfloat16), O.bf16_to_f64(xb)
    z = xd @ w.T
    if r:
        z = z + (xd @ O.f16_to_f64(a).T) @ O.f16_to_f64(b[rows]).T
    bias, gate = rnd(1, n).to(DEV), rnd(2, len(y[0])).to(DEV)
    res = rnd(3, *y.shape).to(DEV).bfloat16()
    y = q2.q2_linear_fused(x, p, s, A, B, bias=bias, gate=gate, residual=res, activation="gelu", gated=gated,
                           out_dtype=torch.bfloat16)
    check(y[:, sel], z, "gelu", gated, bias[torch.from_numpy(rows).to(DEV)], gate[sel], res[:, sel])


def wide_rows(seed, m, k):
    """bf16 bits of rows whose elements differ by up to 2^200 in size, among ordinary ones, and float64 values.
    Every thirteenth row each: one large input; large inputs in the first block only; sizes spread over the whole range;
    two sizes 2^45 apart; the smallest numbers, subnormal ones among them, beside 1; zeros but for the ends; subnormal ones
    alone; two small inputs beside a large one; one that the scale of the large one keeps in part; one among ordinary ones;
    ordinary ones 2^30 below a large one."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k))
    x[1::13, 5] = 2.0 ** 41
    x[2::13, :128] *= 2.0 ** 60
    x[3::13] *= np.ldexp(1.0, rng.integers(-100, 101, x[3::13].shape))
    x[4::13] *= np.where(rng.random(x[4::13].shape) < 0.02, 2.0 ** 45, 1.0)
    x[5::13] = rng.integers(-300, 301, x[5::13].shape) * 2.0 ** -133
    x[5::13, 7] = 1.0
    x[6::13] = 0.0
    x[6::13, [0, k - 1]] = 2.0 ** 90, 2.0 ** -90
    x[7::13] = rng.integers(-127, 128, x[7::13].shape) * 2.0 ** -133
    x[8::13] = 0.0
    x[8::13, [200, 300, 301]] = 2.0 ** 60, 1.5 * 2.0 ** -20, 1.25 * 2.0 ** -20
    x[9::13] = 0.0
    x[9::13, [300, 200]] = -1.0, 255.0 * 2.0 ** -44           # eight bits, four of them below 2^-40
    if k > 400:
        x[10::13, 400] = 1e-30
    x[11::13] *= 2.0 ** -30
    x[11::13, 5] = 1.0
    xb = I.f32_to_bf16_bits(x.astype(np.float32))
    return xb, O.bf16_to_f64(xb)


def wide_weights(seed, n, k):
    """Device weight, codes and scales: every fifth column has no weight at the large inputs of wide_rows, scales go
    from the smallest subnormal f16 to 2^14."""
    codes = np.random.default_rng(seed).integers(0, 3, (n, k)).astype(np.uint8)
    codes[::5, :128] = 1
    for i, (c0, c1) in zip((200, 300, 400), ((1, 2), (0, 1), (2, 0))):        # nothing at one of two inputs of a row
        if i < k:
            codes[::3, i], codes[1::3, i] = c0, c1
    rng = np.random.default_rng(seed + 1)
    scales = np.ldexp(1.0 + rng.integers(0, 1024, (n, k // 128)) / 1024.0, rng.integers(-14, 14, (n, 1)))
    scales[::7] = rng.integers(1, 1024, scales[::7].shape) * 2.0 ** -24
    scales = scales.astype(np.float32)
    return q2.q2_pack(dev_u8(codes), torch.from_numpy(scales).to(DEV)), codes, scales


def own_terms(x, w, a=None, b=None):
    """x W^T (+ (x A^T) B^T) and the RMS sum of every element's own terms."""
    z, size = x @ w.T, (x * x) @ (w * w).T
    if a is not None:
        z, size = z + (x @ a.T) @ b.T, size + ((x * x) @ (a * a).T) @ (b * b).T
    return z, np.sqrt(size)


# sizes that the kernel for many rows takes, the one between, and the plain one
WIDE = [(1000, 5000, 640, 0), (1100, 4100, 12416, 0), (1100, 4100, 12416, 32), (1100, 4100, 4224, 12),
        (700, 8200, 1152, 24), (300, 16400, 512, 64), (1100, 4100, 512, 100), (60, 9000, 640, 8),
        (200, 3000, 384, 8)]


@pytest.mark.parametrize("m,n,k,r", WIDE)
def test_rows_whose_elements_differ_in_size(m, n, k, r):
    """Every output is held to its own terms: where a weight is zero the input adds nothing, however large it is.
    Products are exact and sums are in fp32, so K 2^-24 of the terms' sum would do; the branch's x A^T has 16 bits.
    Terms below fp32's normal numbers may be lost: K of them.  (Other kernels than the one for many rows take a block's
    sum of x off again, so an input of 2^60 covers the rest of its own block: rows 1 to 5 and 11
    modulo 13 are left out.)"""
    (p, s), codes, scales = wide_weights(361, n, k)
    cols, _ = sample(n, False, 361)
    w = (codes[cols].astype(np.float64) - 1) * np.repeat(scales[cols].astype(np.float64), 128, axis=1)
    xb, x = wide_rows(361, m, k)
    A = B = a = b = None
    if r:
        ab, bb = I.lowrank_factors(361, r, k, n, std=0.05)
        ab[:, :128] = 0                                     # the branch sees none of the first block's large inputs
        A, B = dev_bits(ab, torch.float16), dev_bits(bb, torch.float16)
        a, b = O.f16_to_f64(ab), O.f16_to_f64(bb[cols])
    z, size = own_terms(x, w, a, b)
    got = q2.q2_linear_fused(dev_bits(xb, torch.bfloat16), p, s, A, B)
    assert torch.equal(got, q2.q2_linear_fused(dev_bits(xb, torch.bfloat16), p, s, A, B))
    g = host(got[:, torch.from_numpy(cols).to(DEV)])
    assert np.isfinite(g).all()
    bad = np.abs(g - z) > 1e-3 * size + k * 2.0 ** -126
    if not (n >= 1536 and k >= 512 and m >= 300):
        for i in (1, 2, 3, 4, 5, 11):
            bad[i::13] = False
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, in rows {np.unique(np.argwhere(bad)[:, 0] % 13)} modulo 13"


@pytest.mark.parametrize("m,n,k,r", [(1100, 8200, 640, 0), (400, 16400, 512, 20)])
def test_gated_rows_whose_elements_differ_in_size(m, n, k, r):
    """Both factors of an output held to their own terms."""
    (p, s), codes, scales = wide_weights(364, n, k)
    cols, rows = sample(n, True, 364)
    w = (codes[rows].astype(np.float64) - 1) * np.repeat(scales[rows].astype(np.float64), 128, axis=1)
    xb, x = wide_rows(364, m, k)
    A = B = a = b = None
    if r:
        ab, bb = I.lowrank_factors(364, r, k, n, std=0.05)
        ab[:, :128] = 0
        A, B = dev_bits(ab, torch.float16), dev_bits(bb, torch.float16)
        a, b = O.f16_to_f64(ab), O.f16_to_f64(bb[rows])
    z, size = own_terms(x, w, a, b)
    err, h = 1e-3 * size + k * 2.0 ** -126, len(cols)
    got = host(q2.q2_linear_fused(dev_bits(xb, torch.bfloat16), p, s, A, B, gated=True)[:, torch.from_numpy(cols).to(DEV)])
    ref = z[:, :h] * z[:, h:]
    tol = err[:, :h] * np.abs(z[:, h:]) + err[:, h:] * (np.abs(z[:, :h]) + err[:, :h]) + 2.0 ** -126
    inside = np.abs(ref) + tol < 3e38                       # the others may overflow
    bad = (np.abs(got - ref) > tol)[inside]
    assert inside.mean() > 0.5 and not bad.any(), f"{bad.sum()} of {bad.size} outside"


@pytest.mark.parametrize("counts,n,k", [([400, 0, 500], 10010, 640), ([1, 700, 64], 13000, 512)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_rows_whose_elements_differ_in_size(counts, n, k, gather):
    e, rows = len(counts), sum(counts)
    (p, s), codes, scales = wide_weights(362, e * n, k)
    cols, _ = sample(n, False, 362)
    pick = (np.arange(e)[:, None] * n + cols).ravel()
    w = ((codes[pick].astype(np.float64) - 1) * np.repeat(scales[pick].astype(np.float64), 128, axis=1)).reshape(e, len(cols), k)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xb, x = wide_rows(362, 500 if gather else rows, k)
    index = np.random.default_rng(363).integers(-1, 501, rows).astype(np.int32) if gather else None
    y = q2.q2_linear_grouped(dev_bits(xb, torch.bfloat16), torch.from_numpy(offsets).to(DEV), p.view(e, n, -1),
                             s.view(e, n, -1), row_index=None if index is None else torch.from_numpy(index).to(DEV))
    g = host(y[:, torch.from_numpy(cols).to(DEV)])
    z = F.grouped_products(x, w, offsets, index)
    size = np.sqrt(F.grouped_products(x * x, w * w, offsets, index))
    bad = np.abs(g - z) > 1e-3 * size + k * 2.0 ** -126
    assert np.isfinite(g).all()
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}"


# The tile of the kernel between few and many rows goes by the number of rows and columns.
TILES = [(40, 500), (40, 9000), (100, 7000), (100, 10000), (100, 16000), (100, 19000), (100, 21010), (130, 13000)]


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("k", [640, 2176])
@pytest.mark.parametrize("m,n", TILES)
def test_tiles(fmt, gated, k, m, n):
    dev, w = weights(fmt, 319, n, k)
    cols, rows = sample(n, gated, 319)
    xb, x = acts(319, m, k)
    z = O.bf16_to_f64(xb) @ w[rows].T
    bias = rnd(1, n).to(DEV)
    res = rnd(3, m, n // 2 if gated else n).to(DEV)
    y = fused(fmt)(x, *dev, bias=bias, residual=res, activation="silu", gated=gated)
    sel = torch.from_numpy(cols).to(DEV)
    check(y[:, sel], z, "silu", gated, bias[torch.from_numpy(rows).to(DEV)], residual=res[:, sel])
    yb = fused(fmt)(x, *dev, bias=bias, residual=res, activation="silu", gated=gated, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))


@pytest.mark.parametrize("counts,n,k,gated", [([900], 12000, 512, True), ([300, 0, 1, 799], 10010, 640, False),
                                              ([257, 640], 13000, 1152, True)])
@pytest.mark.parametrize("gather", [False, True])
def test_many_rows_grouped(counts, n, k, gated, gather):
    e, lead, tail = len(counts), 2, 3
    rows = sum(counts) + lead + tail
    codes = np.random.default_rng(317).integers(0, 3, (e * n, k)).astype(np.uint8)
    scales = I.q2_scales(317, e * n, k)
    p, s = q2.q2_pack(dev_u8(codes), torch.from_numpy(scales).to(DEV))
    cols, wr = sample(n, gated, 317)
    pick = (np.arange(e)[:, None] * n + wr).ravel()
    w = ((codes[pick].astype(np.float64) - 1) * np.repeat(scales[pick].astype(np.float64), 128, axis=1)).reshape(e, len(wr), k)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + lead
    x_rows = 401 if gather else rows
    index = None
    if gather:
        index = np.random.default_rng(318).integers(0, x_rows, rows).astype(np.int32)
        index[5::50] = -1
        index[6::50] = x_rows
    xb = spread_rows(318, I.activations_bf16(318, x_rows, k))
    z = F.grouped_products(O.bf16_to_f64(xb), w, offsets, index)
    inside = slice(int(offsets[0]), int(offsets[-1]))
    sel = torch.from_numpy(cols).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        y = torch.full((rows, n // 2 if gated else n), 7.0, device=DEV, dtype=out)
        q2.q2_linear_grouped(dev_bits(xb, torch.bfloat16), torch.from_numpy(offsets).to(DEV), p.view(e, n, -1),
                             s.view(e, n, -1), row_index=None if index is None else torch.from_numpy(index).to(DEV),
                             activation="relu", gated=gated, y=y)
        check(y[inside][:, sel], z[inside], "relu", gated)
        assert (y[:lead] == 7).all() and (y[offsets[-1]:] == 7).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [2, 40, 150])
def test_epilogue(fmt, gated, act, m):
    n, k = 2 * 90, 640
    n_out = n // 2 if gated else n
    dev, w = weights(fmt, 302, n, k)
    xb, x = acts(302, m, k)
    z = O.bf16_to_f64(xb) @ w.T
    bias, gate = rnd(1, n).to(DEV), rnd(2, n_out).to(DEV)
    res = {torch.float32: rnd(3, m, n_out).to(DEV), torch.bfloat16: rnd(3, m, n_out).to(DEV).bfloat16()}
    for out in (torch.float32, torch.bfloat16):
        for kw in (dict(), dict(bias=bias), dict(bias=bias, gate=gate), dict(residual=res[torch.bfloat16]),
                   dict(bias=bias, gate=gate, residual=res[torch.float32]), dict(gate=gate, residual=res[out])):
            y = fused(fmt)(x, *dev, activation=act, gated=gated, out_dtype=out, **kw)
            assert y.shape == (m, n_out) and y.dtype == out
            check(y, z, act, gated, what=f"{fmt} {act} {gated} {out} {sorted(kw)}", **kw)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_of_wide_weights(fmt, gated, act):
    m, n, k = 70, 2 * 4200, 640
    n_out = n // 2 if gated else n
    dev, w = weights(fmt, 343, n, k)
    xb, x = acts(343, m, k)
    z = O.bf16_to_f64(xb) @ w.T
    bias, gate = rnd(1, n).to(DEV), rnd(2, n_out).to(DEV)
    res = rnd(3, m, n_out).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        for kw in (dict(bias=bias, gate=gate, residual=res), dict(gate=gate, residual=res.bfloat16()), dict(bias=bias)):
            y = fused(fmt)(x, *dev, activation=act, gated=gated, out_dtype=out, **kw)
            check(y, z, act, gated, what=f"{fmt} {act} {gated} {out} {sorted(kw)}", **kw)
        y = kw_res = res.to(out).clone()
        fused(fmt)(x, *dev, activation=act, gated=gated, residual=y, y=y)
        assert y is kw_res
        check(y, z, act, gated, residual=res.to(out), what="in place")


@pytest.mark.parametrize("m,n,k,r", [(1, 300, 512, 4), (16, 70, 256, 33), (50, 200, 384, 32), (150, 300, 640, 64),
                                     (260, 520, 512, 100), (20, 64, 128, 1), (90, 9000, 640, 24), (40, 9000, 512, 7),
                                     (16, 2000, 1152, 200)])
@pytest.mark.parametrize("gated", [False, True])
def test_rank_r_branch(m, n, k, r, gated):
    (p, s), w = weights("q2", 303, n, k)
    xb, x = acts(303, m, k)
    a, b = I.lowrank_factors(303, r, k, n, std=0.05)
    A, B = dev_bits(a, torch.float16), dev_bits(b, torch.float16)
    xd = O.bf16_to_f64(xb)
    z = xd @ w.T + (xd @ O.f16_to_f64(a).T) @ O.f16_to_f64(b).T
    bias = rnd(4, n).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        y = q2.q2_linear_fused(x, p, s, A, B, bias=bias, activation="silu", gated=gated, out_dtype=out)
        check(y, z, "silu", gated, bias=bias, what=f"r={r}")


@pytest.mark.parametrize("m", [1, 70, 900])
def test_outputs_beside_x(m):
    """x, y and the residual one behind the other in one buffer; over each other they are refused."""
    k = n = 4096
    (p, s), _ = weights("q2", 350, n, k)
    buf = rnd(1, 3 * m, n).to(DEV).bfloat16()
    x, y, res = buf[m:2 * m], buf[:m], buf[2 * m:]
    want = q2.q2_linear_fused(x.clone(), p, s, residual=res.clone(), out_dtype=torch.bfloat16)
    assert torch.equal(q2.q2_linear_fused(x, p, s, residual=res, y=y), want)
    assert torch.equal(q2.q2_linear_fused(x, p, s, residual=res, y=res), want)
    keep = buf.clone()
    for y in (x, buf.view(-1)[8:8 + m * n].view(m, n)):
        with pytest.raises(q2.Q2Error, match="overlaps"):
            q2.q2_linear_fused(x, p, s, residual=x, y=y)
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [1, 13, 70, 200])
def test_residual_in_place(fmt, out, m):
    n, k = 136, 512
    dev, w = weights(fmt, 304, n, k)
    xb, x = acts(304, m, k)
    r0 = rnd(5, m, n).to(DEV).to(out)
    y = r0.clone()
    got = fused(fmt)(x, *dev, activation="relu", residual=y, y=y)
    assert got is y
    assert torch.equal(y, fused(fmt)(x, *dev, activation="relu", residual=r0, out_dtype=out))
    check(y, O.bf16_to_f64(xb) @ w.T, "relu", residual=r0)


# one size for each kernel beyond the one for few tiles, the first two with rows of whole 16-byte pieces and without
KERNELS = [(60, 9000, 640), (60, 9002, 640), (900, 8200, 512), (900, 8206, 512), (200, 3000, 384)]


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("regime", I.ACT_REGIMES)
@pytest.mark.parametrize("m,n,k", KERNELS)
def test_activation_regimes_of_every_kernel(fmt, regime, m, n, k):
    dev, w = weights(fmt, 347, n, k)
    cols, rows = sample(n, False, 347)
    xb = I.activations_regime_bf16(347, m, k, regime)
    y = fused(fmt)(dev_bits(xb, torch.bfloat16), *dev)
    check(y[:, torch.from_numpy(cols).to(DEV)], O.bf16_to_f64(xb) @ w[rows].T, what=regime)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", KERNELS)
def test_epilogue_in_place_of_every_kernel(fmt, gated, act, m, n, k):
    dev, w = weights(fmt, 348, n, k)
    cols, rows = sample(n, gated, 348)
    sel, wsel = torch.from_numpy(cols).to(DEV), torch.from_numpy(rows).to(DEV)
    n_out = n // 2 if gated else n
    xb, x = acts(348, m, k)
    z = O.bf16_to_f64(xb) @ w[rows].T
    bias, gate, res = rnd(1, n).to(DEV), rnd(2, n_out).to(DEV), rnd(3, m, n_out).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        r0 = res.to(out)
        y = r0.clone()
        assert fused(fmt)(x, *dev, bias=bias, gate=gate, activation=act, gated=gated, residual=y, y=y) is y
        check(y[:, sel], z, act, gated, bias[wsel], gate[sel], r0[:, sel], what="in place")
        other = torch.bfloat16 if out == torch.float32 else torch.float32
        assert torch.equal(y, fused(fmt)(x, *dev, bias=bias, gate=gate, activation=act, gated=gated, residual=r0,
                                         out_dtype=out))
        y = fused(fmt)(x, *dev, activation=act, gated=gated, residual=res.to(other), out_dtype=out)
        check(y[:, sel], z, act, gated, residual=res.to(other)[:, sel], what="mixed types")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k,r", [(200, 3000, 384, 5), (300, 2502, 128, 40), (500, 1300, 256, 200)])
def test_branch_of_the_plain_kernel(gated, m, n, k, r):
    """K below four blocks and more tiles than the kernel for few of them takes."""
    (p, s), w = weights("q2", 349, n, k)
    xb, x = acts(349, m, k)
    a, b = I.lowrank_factors(349, r, k, n, std=0.05)
    xd = O.bf16_to_f64(xb)
    z = xd @ w.T + (xd @ O.f16_to_f64(a).T) @ O.f16_to_f64(b).T
    bias, res = rnd(4, n).to(DEV), rnd(5, m, n // 2 if gated else n).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        y = q2.q2_linear_fused(x, p, s, dev_bits(a, torch.float16), dev_bits(b, torch.float16), bias=bias, residual=res,
                               activation="silu", gated=gated, out_dtype=out)
        check(y, z, "silu", gated, bias=bias, residual=res, what=f"r={r}")


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("m", [1, 7, 40, 200])
@pytest.mark.parametrize("n,k", [(75, 256), (75, 640), (8200, 512)])
def test_unaligned_outputs_and_neighbours(fmt, m, n, k):
    """y and the residual one element past any larger boundary; nothing beside y is written."""
    dev, w = weights(fmt, 305, n, k)
    xb, x = acts(305, m, k)
    z = O.bf16_to_f64(xb) @ w.T
    for out in (torch.float32, torch.bfloat16):
        flat = torch.full((m * n + 40,), 7.0, device=DEV, dtype=out)
        rflat = rnd(6, m * n + 1).to(DEV).to(out)
        y, res = flat[1:1 + m * n].view(m, n), rflat[1:].view(m, n)
        fused(fmt)(x, *dev, residual=res, y=y)
        check(y, z, residual=res)
        assert (flat[:1] == 7).all() and (flat[1 + m * n:] == 7).all()


@pytest.mark.parametrize("m", [1, 20, 200])
def test_empty_sum_and_empty_sizes(m):
    n = 48
    x = torch.empty((m, 0), dtype=torch.bfloat16, device=DEV)
    p, s = torch.empty((n, 0), dtype=torch.uint8, device=DEV), torch.empty((n, 0), dtype=torch.float16, device=DEV)
    bias = rnd(7, n).to(DEV)
    y = q2.q2_linear_fused(x, p, s, bias=bias, activation="relu")
    assert torch.equal(y, bias.clamp(min=0).expand(m, n))
    y = q2.q4_linear_fused(x, p, s, s, bias=bias)
    assert torch.equal(y, bias.expand(m, n))
    (pw, sw), _ = weights("q2", 306, 8, 128)
    assert q2.q2_linear_fused(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), pw, sw).shape == (0, 8)
    assert q2.q2_linear_fused(torch.empty((m, 128), dtype=torch.bfloat16, device=DEV), pw[:0], sw[:0]).shape == (m, 0)


@pytest.mark.parametrize("m", [1, 20])
def test_host_inputs_without_elements(m):
    """Inputs that hold nothing may lie on the host; the outputs do not."""
    n, bias = 48, rnd(7, 48).to(DEV)
    x, p, s = torch.empty((m, 0), dtype=torch.bfloat16), torch.empty((n, 0), dtype=torch.uint8), torch.empty((n, 0)).half()
    for y in (q2.q2_linear_fused(x, p, s, bias=bias), q2.q4_linear_fused(x, p, s, s, bias=bias)):
        assert y.is_cuda and torch.equal(y, bias.expand(m, n))
    dev, _ = weights("q2", 306, n, 128)
    y = q2.q2_linear_grouped(torch.empty((0, 128), dtype=torch.bfloat16), torch.tensor([0, m], dtype=torch.int32, device=DEV),
                             *(t[None] for t in dev), row_index=torch.zeros(m, dtype=torch.int32, device=DEV), bias=bias[None])
    assert y.is_cuda and torch.equal(y, bias.expand(m, n))


@pytest.mark.parametrize("m", [1, 16, 17, 150, 600])
@pytest.mark.parametrize("n,k", [(130, 1280), (6000, 640), (130, 256)])
def test_zero_weights_add_exactly_nothing(m, n, k):
    xb, x = acts(307, m, k)
    codes, scales = np.ones((n, k), np.uint8), I.q2_scales(307, n, k)
    p, s = q2.q2_pack(dev_u8(codes), torch.from_numpy(scales).to(DEV))
    assert (q2.q2_linear_fused(x, p, s) == 0).all()
    p4 = torch.full((n, k // 2), 0x55, dtype=torch.uint8, device=DEV)
    s4 = torch.from_numpy(scales).half().to(DEV)
    assert (q2.q4_linear_fused(x, p4, s4, torch.full_like(s4, 5.0)) == 0).all()


@pytest.mark.parametrize("regime", I.ACT_REGIMES)
@pytest.mark.parametrize("m", [3, 80, 300])
def test_activation_regimes(regime, m):
    n, k = 100, 512
    (p, s), w = weights("q2", 308, n, k)
    xb = I.activations_regime_bf16(308, m, k, regime)
    check(q2.q2_linear_fused(dev_bits(xb, torch.bfloat16), p, s), O.bf16_to_f64(xb) @ w.T, what=regime)


@pytest.mark.parametrize("m", [3, 80, 300])
def test_extreme_scales_and_wide_rows(m):
    """Scales from subnormal to near the f16 maximum, and rows whose elements span the bf16 range around 1."""
    n, k = 96, 640
    codes = I.q2_codes(309, n, k)
    rng = np.random.default_rng(309)
    scales = np.ldexp(1.0 + rng.integers(0, 1024, (n, k // 128)) / 1024.0, rng.integers(-14, 15, (n, 1)))
    scales[::7] = rng.integers(1, 1024, scales[::7].shape) * 2.0 ** -24            # subnormal rows
    scales = scales.astype(np.float16).astype(np.float32)
    p, s = q2.q2_pack(dev_u8(codes), torch.from_numpy(scales).to(DEV))
    w = O.unpack_q2(*O.pack_q2(codes, scales)).astype(np.float64)
    xf = rng.standard_normal((m, k)) * np.ldexp(1.0, rng.integers(-30, 1, (m, k)))
    xb = I.f32_to_bf16_bits(xf.astype(np.float32))
    z = O.bf16_to_f64(xb) @ w.T
    got = host(q2.q2_linear_fused(dev_bits(xb, torch.bfloat16), p, s))
    # columns have scales of their own: each is held to the bar of its own terms
    bar = 1e-3 * np.sqrt((O.bf16_to_f64(xb) ** 2) @ (w ** 2).T)
    assert (np.abs(got - z) <= bar).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
def test_offsets_beyond_32_bits(fmt):
    """More than 2^32 output elements' bytes: row and element indices beyond 31 bits."""
    m, n, k = 70001, 32770, 128
    dev, w = weights(fmt, 310, n, k)
    xb, x = acts(310, m, k)
    y = fused(fmt)(x, *dev, out_dtype=torch.bfloat16)
    assert m * n > 2 ** 31
    rows = np.array([0, 1, 31999, 65535, 65537, m - 2, m - 1])
    z = O.bf16_to_f64(xb[rows]) @ w.T
    check(y[torch.from_numpy(rows).to(DEV)], z)


def test_more_than_32_bits_of_threads_one_row():
    """2^24 workgroups of 256 threads and a few more: every column is the sum of x or its negative."""
    n, k = 2 ** 29 + 70, 128
    p = torch.full((n, k // 4), 0xAA, dtype=torch.uint8, device=DEV)          # codes 2
    p[n // 2:] = 0                                                            # codes 0
    x = torch.ones((1, k), device=DEV, dtype=torch.bfloat16)
    y = torch.zeros((1, n), device=DEV)
    q2.q2_linear_fused(x, p, torch.ones((n, 1), device=DEV, dtype=torch.float16), y=y)
    assert (y[0, :n // 2] == k).all() and (y[0, n // 2:] == -k).all()
    del p, y
    torch.cuda.empty_cache()


def test_more_than_32_bits_of_threads_many_rows():
    """More than 2^24 tiles of 32 x 64."""
    m, n, k = 2 ** 20 + 40, 2 ** 15, 128
    dev, w = weights("q2", 346, n, k)
    xb, x = acts(346, 4096, k)
    row = torch.arange(m, device=DEV) % 4096
    y = torch.full((m, n), 7.0, device=DEV, dtype=torch.bfloat16)
    q2.q2_linear_fused(x[row], *dev, y=y)
    want = y[:4096].clone()
    check(want[:64], O.bf16_to_f64(xb[:64]) @ w.T)
    for lo in range(0, m, 4096):
        part = y[lo:lo + 4096]
        assert torch.equal(part, want[:len(part)])
    del y
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# grouped
# ---------------------------------------------------------------------------

def group_case(fmt, counts, n, k, x_rows=None, seed=320, lead=0, tail=0):
    """Device weights, float64 weights, offsets, x (bits and tensor) and a row index of ragged groups."""
    e = len(counts)
    dev, w = weights(fmt, seed, e * n, k)
    dev = tuple(t.view(e, n, -1) for t in dev)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + lead
    rows = int(offsets[-1]) + tail
    index = None
    if x_rows is not None:
        index = np.random.default_rng(seed).integers(0, x_rows, rows).astype(np.int32)
    xb, x = acts(seed, rows if x_rows is None else x_rows, k)
    return dev, w.reshape(e, n, k), offsets, xb, x, index


COUNTS = [[5], [0, 3, 0, 0, 1], [17, 0, 40, 1, 33], [1] * 8, [0] * 3 + [130], [300, 2, 0, 64, 129],
          [2, 0, 1] * 25, [0, 0]]


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k", [384, 640])
def test_grouped(fmt, counts, gather, k):
    n = 2 * 45
    lead, tail = (0, 0) if gather else (3, 5)
    dev, w, offsets, xb, x, index = group_case(fmt, counts, n, k, x_rows=37 if gather else None, lead=lead, tail=tail)
    z = F.grouped_products(O.bf16_to_f64(xb), w, offsets, index)
    rows, inside = len(z), slice(int(offsets[0]), int(offsets[-1]))
    expert = np.repeat(np.arange(len(counts)), counts)
    off = torch.from_numpy(offsets).to(DEV)
    idx = None if index is None else torch.from_numpy(index).to(DEV)
    bias = rnd(8, len(counts), n).to(DEV)
    for act, gated, out, b in (("none", False, torch.float32, None), ("silu", True, torch.bfloat16, bias),
                               ("gelu", False, torch.float32, bias), ("relu", True, torch.float32, None)):
        y = torch.full((rows, n // 2 if gated else n), 7.0, device=DEV, dtype=out)
        grouped(fmt)(x, off, *dev, row_index=idx, bias=b, activation=act, gated=gated, y=y)
        rb = None if b is None else b[torch.from_numpy(expert).to(DEV)]
        if sum(counts):
            check(y[inside], z[inside], act, gated, bias=rb, what=f"{fmt} {counts} {act}")
        assert (y[:offsets[0]] == 7).all() and (y[offsets[-1]:] == 7).all(), "a row of no expert was written"


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("rows_per", [2, 60])
def test_grouped_rows_equal_the_experts_own_linears(fmt, rows_per):
    """Every expert's rows against the fused linear on its own weight (other launch shapes, so within the bar)."""
    counts = [rows_per, 0, 2 * rows_per, 1]
    n, k = 200, 512
    dev, w, offsets, xb, x, _ = group_case(fmt, counts, n, k)
    y = grouped(fmt)(x, torch.from_numpy(offsets).to(DEV), *dev, activation="gelu_tanh")
    for e in range(len(counts)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            z = O.bf16_to_f64(xb[lo:hi]) @ w[e].T
            check(y[lo:hi], z, "gelu_tanh")
            check(fused(fmt)(x[lo:hi], *(t[e] for t in dev), activation="gelu_tanh"), z, "gelu_tanh")


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("rows", [4, 200])
@pytest.mark.parametrize("k", [256, 1152])
def test_grouped_index_outside_x_reads_zeros(fmt, rows, k):
    n = 64
    counts = [rows, rows]
    dev, w, offsets, xb, x, index = group_case(fmt, counts, n, k, x_rows=9)
    index[::3] = np.array([-1, 9, 2 ** 31 - 1, -2 ** 31] * rows, np.int32)[:len(index[::3])]
    z = F.grouped_products(O.bf16_to_f64(xb), w, offsets, index)
    assert (z[::3] == 0).all()
    y = grouped(fmt)(x, torch.from_numpy(offsets).to(DEV), *dev, row_index=torch.from_numpy(index).to(DEV))
    check(y, z)
    assert (y[::3] == 0).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("bad", [[5, 40, 20, 64], [-7, 20, 90, 64], [0, 2 ** 31 - 1, -2 ** 31, 50], [64, 0, 64, 0]])
@pytest.mark.parametrize("k", [128, 640])
def test_grouped_bad_offsets_stay_inside(fmt, bad, k):
    """Offsets that decrease or leave [0, R]: only rows of y are written, the rest of its storage is not."""
    rows, n = 64, 40
    dev, _, _, _, x, _ = group_case(fmt, [rows, 0, 0], n, k)
    flat = torch.full((3 * rows * n,), 7.0, device=DEV)
    y = flat[rows * n:2 * rows * n].view(rows, n)
    grouped(fmt)(x, torch.tensor(bad, dtype=torch.int32, device=DEV), *dev, y=y)
    torch.cuda.synchronize()
    assert (flat[:rows * n] == 7).all() and (flat[2 * rows * n:] == 7).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("counts", [[60, 0, 90, 45, 100], [300, 150, 0, 400]])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k", [640, 2176])
def test_grouped_wide(fmt, counts, gather, k):
    """Enough columns for the wider tiles; rows of no expert hold NaN, which no other row may read."""
    n, lead, tail = 1320, 3, 5
    dev, w, offsets, xb, x, index = group_case(fmt, counts, n, k, x_rows=77 if gather else None, lead=lead, tail=tail)
    if not gather:
        x[:lead] = np.nan
        x[-tail:] = np.nan
    else:
        index[:lead] = 2 ** 30
        index[-tail:] = -5
    z = F.grouped_products(O.bf16_to_f64(xb), w, offsets, index)
    inside = slice(int(offsets[0]), int(offsets[-1]))
    expert = torch.from_numpy(np.repeat(np.arange(len(counts)), counts)).to(DEV)
    bias = rnd(8, len(counts), n).to(DEV)
    idx = None if index is None else torch.from_numpy(index).to(DEV)
    for gated, out in ((False, torch.float32), (True, torch.bfloat16), (True, torch.float32)):
        y = torch.full((len(z), n // 2 if gated else n), 7.0, device=DEV, dtype=out)
        grouped(fmt)(x, torch.from_numpy(offsets).to(DEV), *dev, row_index=idx, bias=bias, activation="silu",
                     gated=gated, y=y)
        check(y[inside], z[inside], "silu", gated, bias=bias[expert])
        assert (y[:lead] == 7).all() and (y[-tail:] == 7).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("m,n,k", [(3, 200, 512), (40, 300, 640), (100, 16000, 640), (50, 70, 256), (900, 8200, 512)])
def test_non_finite_rows_stay_alone(fmt, m, n, k):
    """A row of x that holds an infinity or a NaN has no finite product; every other row is what it is without it."""
    dev, _ = weights(fmt, 341, n, k)
    _, x = acts(341, m, k)
    want = fused(fmt)(x, *dev)
    bad = x.clone()
    bad[1, 5], bad[2, k - 1] = np.inf, np.nan
    got = fused(fmt)(bad, *dev)
    assert not torch.isfinite(got[1:3]).any()
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    assert torch.equal(got[keep], want[keep]) and torch.isfinite(want).all()


# of an activation: the range on which its value is a normal number, the exact value, and the size of the argument of its
# exponential, whose rounding the value takes over
TAILS = {"gelu": (13.0, lambda v: v * scipy.special.ndtr(v), lambda v: v * v / 2),
         "gelu_tanh": (9.5, lambda v: v * scipy.special.expit(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)),
                       lambda v: math.sqrt(8 / math.pi) * np.abs(v + 0.044715 * v ** 3)),
         "silu": (80.0, lambda v: v * scipy.special.expit(v), np.abs)}


@pytest.mark.parametrize("act", TAILS)
@pytest.mark.parametrize("m,n,k", [(2, 16000, 128), (40, 16000, 640), (100, 16001, 256), (900, 16000, 512)])
def test_activations_relative_to_their_values(act, m, n, k):
    """The bias alone (x is 0): every value to a few ulps of itself, also where it is tiny, as a gated factor multiplies
    it.  Of an exponential of argument u four roundings of u (three in u, one in the exponential's base) add
    4 |u| 2^-24; the exponential, a reciprocal, a polynomial of positive value and four products sixteen more."""
    most, exact, argument = TAILS[act]
    dev, _ = weights("q2", 345, 2 * n, k)
    v = torch.linspace(-most, most, n)
    bias = torch.cat([v, torch.full((n,), 3.0)]).to(DEV)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    vd = v.double().numpy()
    tol = 2.0 ** -24 * (4 * argument(vd) + 16) * np.abs(exact(vd)) + 2.0 ** -126
    got = host(q2.q2_linear_fused(x, *dev, bias=bias, activation=act, gated=True)[-1])
    assert (np.abs(got / 3 - exact(vd)) <= tol).all()
    got = host(q2.q2_linear_fused(x, *(t[:n] for t in dev), bias=bias[:n].contiguous(), activation=act)[-1])
    assert (np.abs(got - exact(vd)) <= tol).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(3, 200, 512), (40, 8206, 640), (100, 16000, 640), (100, 2002, 256), (900, 8200, 512)])
def test_activations_keep_a_nan(fmt, act, m, n, k):
    """A row of x with a NaN is NaN in every output, behind every activation, gated or not, in either column order."""
    dev, _ = weights(fmt, 344, n, k)
    _, x = acts(344, m, k)
    x[2, k - 1] = np.nan
    for gated in (False, True):
        for out in (torch.float32, torch.bfloat16):
            y = fused(fmt)(x, *dev, activation=act, gated=gated, out_dtype=out)
            assert torch.isnan(y[2]).all() and torch.isfinite(y[:2]).all() and torch.isfinite(y[3:]).all()
    off = torch.tensor([0, 2, m], dtype=torch.int32, device=DEV)
    y = grouped(fmt)(x, off, *(torch.stack([t, t]) for t in dev), activation=act)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[:2]).all() and torch.isfinite(y[3:]).all()


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("rows,k", [(3, 128), (3, 640), (60, 256), (200, 640), (1100, 512)])
def test_grouped_without_a_row_of_x(fmt, rows, k):
    """An index into no rows: every product is empty, the epilogue remains."""
    n = 2400
    dev, _ = weights(fmt, 342, 2 * n, k)
    bias = rnd(9, 2, n).to(DEV)
    y = grouped(fmt)(torch.empty((0, k), device=DEV, dtype=torch.bfloat16),
                     torch.tensor([0, 1, rows], dtype=torch.int32, device=DEV), *(t.view(2, n, -1) for t in dev),
                     row_index=torch.zeros(rows, dtype=torch.int32, device=DEV), bias=bias, activation="relu")
    assert torch.equal(y[:1], bias[:1].clamp(min=0)) and torch.equal(y[1:], bias[1:].clamp(min=0).expand(rows - 1, n))


@pytest.mark.parametrize("m", [1, 30])
def test_branch_of_an_empty_sum(m):
    n, r = 48, 4
    e = lambda *shape, dtype=torch.float16: torch.empty(shape, dtype=dtype, device=DEV)      # noqa: E731
    y = q2.q2_linear_fused(e(m, 0, dtype=torch.bfloat16), e(n, 0, dtype=torch.uint8), e(n, 0), e(r, 0),
                           torch.ones((n, r), device=DEV).half())
    assert y.shape == (m, n) and (y == 0).all()


# ---------------------------------------------------------------------------
# streams, graphs, repeatability
# ---------------------------------------------------------------------------

def stream_cases():
    """(name, call(x) -> tensor, x) over the variants: few rows, many rows, branch, grouped."""
    out = []
    (p, s), _ = weights("q2", 330, 256, 512)
    dev4, _ = weights("q4", 330, 256, 512)
    a, b = I.lowrank_factors(330, 8, 512, 256)
    A, B = dev_bits(a, torch.float16), dev_bits(b, torch.float16)
    for m in (2, 40, 300):
        _, x = acts(331, m, 512)
        out.append((f"q2 {m}", lambda x: q2.q2_linear_fused(x, p, s, A, B, activation="silu", gated=True), x))
        out.append((f"q4 {m}", lambda x: q2.q4_linear_fused(x, *dev4, activation="gelu"), x))
    (pw, sw), _ = weights("q2", 333, 12300, 512)
    Bw = dev_bits(I.lowrank_factors(330, 8, 512, 12300)[1], torch.float16)
    dev4w, _ = weights("q4", 333, 9000, 512)
    for m in (100, 300):
        _, x = acts(331, m, 512)
        out.append((f"q2 wide {m}", lambda x: q2.q2_linear_fused(x, pw, sw, A, Bw, activation="silu", gated=True), x))
        out.append((f"q4 wide {m}", lambda x: q2.q4_linear_fused(x, *dev4w, activation="gelu"), x))
    _, x = acts(331, 900, 512)
    out.append(("q2 900", lambda x: q2.q2_linear_fused(x, pw, sw, A, Bw, activation="silu"), x))
    for counts in ([1, 0, 2, 1], [100, 0, 37, 163]):
        dev, _, offsets, _, x, _ = group_case("q2", counts, 64, 512, seed=332)
        off = torch.from_numpy(offsets).to(DEV)
        out.append((f"grouped {sum(counts)}", lambda x, off=off, dev=dev: q2.q2_linear_grouped(x, off, *dev), x))
    return out


def test_repeatable_on_a_busy_side_stream():
    for name, call, x in stream_cases():
        want = call(x)
        side = torch.cuda.Stream()
        late = torch.zeros_like(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big = torch.randn(4096, 4096, device=DEV)
            for _ in range(4):
                big = big @ big.clamp(-1e-3, 1e-3)
            late.copy_(x)                                   # written late on this stream
            got = call(late)
        side.synchronize()
        assert torch.equal(got, want), name


def test_graph_replays_equal_eager_calls():
    for name, call, x in stream_cases():
        static = x.clone()
        call(static)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            call(static)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                y = call(static)
        for i in range(3):
            new = torch.roll(x, i + 1, dims=1).contiguous()
            want = call(new)                                # eager work between the replays
            static.copy_(new)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), f"{name}: replay {i}"


def test_two_graphs_and_an_eager_call_at_once():
    """Two captured calls replayed on two streams while a third runs eagerly: each has scratch of its own."""
    for name, call, x in stream_cases():
        streams, xs, ys, graphs = [torch.cuda.Stream() for _ in range(2)], [], [], []
        want = [call(torch.roll(x, i, dims=1).contiguous()) for i in range(3)]
        torch.cuda.synchronize()
        for i in range(2):
            xs.append(torch.roll(x, i, dims=1).contiguous())
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.stream(streams[i]), torch.cuda.graph(graphs[i], stream=streams[i]):
                ys.append(call(xs[i]))
        third = torch.roll(x, 2, dims=1).contiguous()
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
            eager = call(third)
            torch.cuda.synchronize()
            assert torch.equal(eager, want[2]) and torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1]), name


def test_refusals():
    (p, s), _ = weights("q2", 340, 7, 128)
    _, x = acts(340, 3, 128)
    with pytest.raises(ValueError, match="activation"):
        q2.q2_linear_fused(x, p, s, activation="swish")
    with pytest.raises(ValueError, match="halves"):
        q2.q2_linear_fused(x, p, s, gated=True)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        q2.q2_linear_fused(x, p, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="residual"):
        q2.q2_linear_fused(x, p, s, residual=torch.zeros(3, 8, device=DEV))
    with pytest.raises(ValueError, match="bias"):
        q2.q2_linear_fused(x, p, s, bias=torch.zeros(7, device=DEV).double())
    with pytest.raises(ValueError, match="come together"):
        q2.q2_linear_fused(x, p, s, A=torch.zeros((4, 128), device=DEV).half())
    with pytest.raises(ValueError, match="offsets"):
        q2.q2_linear_grouped(x, torch.zeros(3, device=DEV, dtype=torch.int32), p[None], s[None])
    with pytest.raises(ValueError, match="device tensor"):
        q2.q2_linear_fused(x.cpu(), p, s)
