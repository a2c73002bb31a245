"""GPU tests of the router and the combination against the float64 oracle, and of
a run of them with the grouped linears between, as they are used together.

Whole numbers are equal.  A weight is a quotient of fp32 exponentials of
differences d of logits: the hardware's exp is off by about an ulp plus |d|
half-ulps of its argument, the sum of E terms by E / 2 ulps: relative
2^-24 (2 (|d| + 2) + E).  A combination of k terms is off by (k + 1) / 2 ulps of
the sum of their magnitudes, and the output type adds half a step.
"""
import numpy as np
import pytest
import torch

import oracle.fused_oracle as F
import oracle.q2_oracle as O
import ternary_weight_quantized_q2_amd as q2
from tests.test_fused_gpu import check, group_case, host, rnd
from tests.test_parity_gpu import DEV, acts, q2_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU parity tests need a GPU; they must not be skipped silently"
    torch.cuda.set_device(0)
    q2.load()
    yield


def check_route(logits, k, renorm):
    e = logits.shape[1]
    got = q2.q2_route(logits.to(DEV), k, renormalize=renorm)
    want = F.route(logits.double().numpy(), k, renorm)
    for name, g, w in zip(got._fields, got, want):
        g = g.cpu().numpy()
        if name == "weight":
            with np.errstate(divide="ignore"):
                d = np.where(w > 0, -np.log(np.where(w > 0, w, 1.0)), 104.0)     # at least the exponent of the weight
            tol = w * 2.0 ** -24 * (2 * (np.minimum(d, 104) + 2) + e + 2 * d) + 2.0 ** -126
            assert (np.abs(g - w) <= tol).all(), name
        else:
            assert np.array_equal(g, w), name
    return got


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (64, 8, 2), (65, 8, 2), (63, 130, 4), (200, 256, 8),
                                   (129, 70, 33), (500, 16, 1), (70, 1024, 64), (130, 512, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(t, e, k, dtype, renorm):
    check_route((rnd(t + e, t, e) * 3).to(dtype), k, renorm)


@pytest.mark.parametrize("t", [1, 61, 130])
@pytest.mark.parametrize("e,k", [(64, 8), (61, 17), (100, 16), (128, 17), (130, 8), (256, 30), (300, 5), (1000, 12)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_ties_at_every_size(t, e, k, renorm):
    """Few values, many of them masked: equal logits go to the lower expert wherever the experts are held."""
    v = torch.randint(-2, 3, (t, e), generator=torch.Generator().manual_seed(3)).float()
    v[torch.rand((t, e), generator=torch.Generator().manual_seed(4)) < 0.6] = -np.inf
    v[t // 2, 3:] = -np.inf
    v[t // 3, : e // 2] = np.nan
    check_route(v, k, renorm)
    check_route(v.bfloat16(), k, renorm)


@pytest.mark.parametrize("t", [40, 300])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_ties_masks_and_extremes(t, renorm):
    e, k = 24, 4
    v = torch.randint(-2, 3, (t, e), generator=torch.Generator().manual_seed(1)).float()      # many ties
    v[0] = 0.0
    v[0, ::2] = -0.0                                       # equal to +0
    v[1] = -np.inf                                         # a padding token
    v[2] = np.nan
    v[3, 3:] = -np.inf                                     # fewer experts than k
    v[4] = torch.finfo(torch.float32).min                  # the type's lowest value is a logit like any other
    v[5, 5] = torch.finfo(torch.float32).max
    v[6, [4, 9]] = np.inf
    v[7, ::3] = np.nan
    v[8] = -np.inf
    v[8, 23] = -1e30
    v[9, :20] = torch.finfo(torch.float32).min
    got = check_route(v, k, renorm)
    assert (got.expert[1] == -1).all() and (got.weight[1:3] == 0).all()
    assert got.expert[6, :2].tolist() == [4, 9] and got.weight[6, :2].tolist() == [0.5, 0.5]
    check_route(torch.full((t, e), -np.inf), k, renorm)    # nobody has a row
    check_route(torch.zeros((t, e)), k, renorm)            # everybody the same experts


def test_route_many_tokens():
    """More tokens than 1024 workgroups of one chunk hold: several chunks each, the last ones partly empty."""
    v = torch.randint(0, 50, (70001, 6), generator=torch.Generator().manual_seed(2)).float()
    v[::5] = -np.inf
    check_route(v, 2, True)


@pytest.mark.parametrize("t", [1023 * 65536 + 1, 2 ** 26])
@pytest.mark.parametrize("e,k", [(1, 1), (2, 2)])
def test_route_of_the_most_tokens(t, e, k):
    """Every token chooses every expert: expert j's rows are all tokens in their order.  (t, e, k) up to the largest t."""
    logits = torch.zeros((t, e), device=DEV, dtype=torch.bfloat16)
    got = q2.q2_route(logits, k)
    assert got.offsets.tolist() == [j * t for j in range(e + 1)]
    token = torch.arange(t, device=DEV, dtype=torch.int32)
    for j in range(e):
        assert torch.equal(got.expert[:, j], torch.full_like(token, j))
        assert torch.equal(got.slot[:, j], token + j * t) and torch.equal(got.row_token[j * t:(j + 1) * t], token)
    assert (got.weight == 1 / k).all()


def test_route_of_the_most_tokens_to_one_expert():
    """The last workgroups' tokens all choose one expert of three, most of the others' none."""
    t = 2 ** 26
    logits = torch.zeros((t, 3), device=DEV, dtype=torch.bfloat16)
    logits[:t // 2] = -np.inf
    logits[t // 2:, 1] = 1
    logits[5, 2] = 0
    got = q2.q2_route(logits, 1)
    rows = t // 2
    assert got.offsets.tolist() == [0, 0, rows, rows + 1]
    assert torch.equal(got.slot[t // 2:, 0], torch.arange(rows, device=DEV, dtype=torch.int32))
    assert torch.equal(got.row_token[:rows], torch.arange(rows, t, device=DEV, dtype=torch.int32))
    assert got.slot[5].item() == rows and got.row_token[rows].item() == 5 and (got.row_token[rows + 1:] == -1).all()


def test_route_of_no_tokens():
    got = q2.q2_route(torch.empty((0, 12), device=DEV), 3)
    assert got.offsets.tolist() == [0] * 13 and got.expert.shape == (0, 3) and got.row_token.numel() == 0


def test_host_inputs_without_elements():
    """Inputs that hold nothing may lie on the host; the outputs do not."""
    got = q2.q2_route(torch.empty((0, 12)), 3)
    assert all(t.is_cuda for t in got) and got.offsets.tolist() == [0] * 13
    res = rnd(1, 3, 8).to(DEV)
    y = q2.q2_combine(torch.empty((0, 8)), torch.zeros((3, 2), dtype=torch.int32, device=DEV),
                      torch.ones((3, 2), device=DEV), residual=res)
    assert y.is_cuda and torch.equal(y, res)
    assert torch.equal(q2.q2_combine(torch.empty((0, 8)), torch.empty((3, 0), dtype=torch.int32), torch.empty((3, 0)),
                                     residual=res), res)


def test_route_refusals():
    x = torch.zeros((2, 8), device=DEV)
    for k in (0, 9, -1, 10 ** 12):
        with pytest.raises(q2.Q2Error):
            q2.q2_route(x, k)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        q2.q2_route(x.double(), 2)
    with pytest.raises(q2.Q2Error):
        q2.q2_route(torch.zeros((1, 1025), device=DEV), 2)
    with pytest.raises(ValueError, match="contiguous"):
        q2.q2_route(torch.zeros((8, 8), device=DEV).t()[1:, ::2], 2)


def check_combine(t, k, n, r, zt, rt, out, seed=0, slot=None):
    g = np.random.default_rng(seed)
    z = rnd(seed, r, n).to(zt)
    if slot is None:
        slot = g.integers(-1, r, (t, k)).astype(np.int32)
    weight = rnd(seed + 1, t, k)
    res = None if rt is None else rnd(seed + 2, t, n).to(rt)
    y = q2.q2_combine(z.to(DEV), torch.from_numpy(slot).to(DEV), weight.to(DEV),
                      residual=None if res is None else res.to(DEV), out_dtype=out)
    assert y.dtype == out
    zd, wd, rd = host(z), host(weight), host(res)
    ref = F.combine(zd, slot, wd, rd)
    size = F.combine(np.abs(zd), slot, np.abs(wd), None if rd is None else np.abs(rd))
    tol = (k + 1) * 2.0 ** -24 * size
    tol += (np.abs(ref) + tol) * torch.finfo(out).eps / 2
    assert (np.abs(host(y) - ref) <= tol).all()


@pytest.mark.parametrize("t,k,n,r", [(1, 8, 2048, 8), (5, 1, 1, 3), (3, 2, 8, 4), (7, 4, 37, 20), (130, 3, 264, 300),
                                     (2, 64, 100, 50), (4, 0, 16, 2), (9, 3, 518, 30), (5, 2, 257, 9), (3, 2, 1030, 7)])
@pytest.mark.parametrize("zt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rt", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_combine(t, k, n, r, zt, rt, out):
    check_combine(t, k, n, r, zt, rt, out)


def test_combine_slots_outside_and_repeated():
    slot = np.array([[-1, 5, 2 ** 31 - 1], [0, 0, 0], [4, -2 ** 31, 4], [-1, -1, -1]], np.int32)
    check_combine(4, 3, 24, 5, torch.bfloat16, torch.float32, torch.float32, slot=slot)
    check_combine(4, 3, 24, 0, torch.bfloat16, torch.float32, torch.float32, slot=slot)        # no rows at all


@pytest.mark.parametrize("n", [64, 37])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_combine_in_place_and_unaligned(n, dt):
    t, k = 9, 3
    z, w = rnd(3, 30, n).to(DEV), rnd(4, t, k).to(DEV)
    slot = torch.randint(0, 30, (t, k), device=DEV, dtype=torch.int32)
    r0 = rnd(5, t, n).to(DEV).to(dt)
    want = q2.q2_combine(z, slot, w, residual=r0, out_dtype=dt)
    flat = torch.full((t * n + 9,), 7.0, device=DEV, dtype=dt)
    y = flat[1:1 + t * n].view(t, n)
    y.copy_(r0)
    assert q2.q2_combine(z, slot, w, residual=y, y=y) is y
    assert torch.equal(y, want) and (flat[:1] == 7).all() and (flat[1 + t * n:] == 7).all()


def test_combine_beyond_32_bits():
    """z of more than 2^31 elements, its last rows used."""
    n, r = 65536, 33000
    z = torch.zeros((r, n), dtype=torch.bfloat16, device=DEV)
    z[-1], z[0] = 3.0, 1.0
    y = q2.q2_combine(z, torch.tensor([[r - 1, 0], [0, 0]], dtype=torch.int32, device=DEV),
                      torch.tensor([[2.0, 1.0], [1.0, 0.5]], device=DEV))
    assert (y[0] == 7).all() and (y[1] == 1.5).all()


@pytest.mark.parametrize("t,n,out", [(2 ** 26 + 9, 1, torch.float32), (2 ** 26 + 9, 2, torch.bfloat16),
                                     (2 ** 23 + 1, 4096, torch.bfloat16)])
def test_combine_of_more_than_32_bits_of_threads(t, n, out):
    """Every token's row is its weight, all of them written."""
    weight = (torch.arange(t, device=DEV) % 251).float().view(t, 1)
    y = torch.full((t, n), -1.0, device=DEV, dtype=out)
    q2.q2_combine(torch.ones((1, n), device=DEV), torch.zeros((t, 1), device=DEV, dtype=torch.int32), weight, y=y)
    for lo in range(0, t, 2 ** 20):                         # whole numbers below 2^8 are exact in bf16
        assert (y[lo:lo + 2 ** 20] == weight[lo:lo + 2 ** 20]).all()
    del y
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# together: an expert layer with its router, from logits to the residual stream
# ---------------------------------------------------------------------------

def expert_layer(x, logits, k, w1, w2, y):
    """y += the experts' gated layers of x."""
    r = q2.q2_route(logits, k)
    h = q2.q2_linear_grouped(x, r.offsets, *w1, row_index=r.row_token, activation="silu", gated=True,
                             out_dtype=torch.bfloat16)
    z = q2.q2_linear_grouped(h, r.offsets, *w2, out_dtype=torch.bfloat16)
    return r, h, z, q2.q2_combine(z, r.slot, r.weight, residual=y, y=y)


@pytest.mark.parametrize("t,e,k,hidden,inner", [(1, 8, 2, 256, 128), (23, 6, 3, 128, 256), (150, 4, 2, 384, 256)])
def test_expert_layer(t, e, k, hidden, inner):
    w1, w1d, _, xb, x, _ = group_case("q2", [t] + [0] * (e - 1), 2 * inner, hidden, seed=350)
    w2, w2d, _, _, _, _ = group_case("q2", [1] * e, hidden, inner, seed=351)
    logits = rnd(9, t, e)
    logits[t // 2] = -np.inf                               # one padding token (the only one when t == 1)
    y0 = rnd(10, t, hidden).to(DEV).bfloat16()
    r, h, z, y = expert_layer(x, logits.to(DEV), k, w1, w2, y0.clone())
    expert, weight, offsets, token, slot = F.route(logits.double().numpy(), k, True)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets) and np.array_equal(r.row_token.cpu().numpy(), token)
    rows = int(offsets[-1])
    if rows:
        zh = F.grouped_products(O.bf16_to_f64(xb), w1d, offsets, token)[:rows]
        check(h[:rows], zh, "silu", True)
        hd = np.zeros(h.shape)
        hd[:rows] = host(h[:rows])
        check(z[:rows], F.grouped_products(hd, w2d, offsets)[:rows])
    zd = np.zeros(z.shape)
    zd[:rows] = host(z[:rows])
    ref = F.combine(zd, slot, weight, host(y0))
    size = F.combine(np.abs(zd), slot, weight, np.abs(host(y0)))
    assert (np.abs(host(y) - ref) <= 2.0 ** -20 * size + np.abs(ref) * torch.finfo(torch.bfloat16).eps / 2).all()
    pad = t // 2
    assert torch.equal(y[pad], y0[pad])                    # the padding token's stream is untouched


def test_expert_layer_in_a_graph():
    t, e, k = 90, 6, 2
    w1, _, _, _, x, _ = group_case("q2", [t] + [0] * (e - 1), 256, 256, seed=352)
    w2, _, _, _, _, _ = group_case("q2", [1] * e, 256, 128, seed=353)
    logits, y = rnd(11, t, e).to(DEV), torch.zeros((t, 256), device=DEV)
    expert_layer(x, logits, k, w1, w2, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            expert_layer(x, logits, k, w1, w2, y)
    for i in range(3):
        logits.copy_(rnd(12 + i, t, e))
        y.fill_(i)
        want = expert_layer(x, logits, k, w1, w2, y.clone())[3]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"


def test_dense_gated_layer_through_both_linears():
    """The two fused linears of a gated layer, bf16 between, onto the residual stream."""
    m, hidden, inner = 70, 256, 384
    p1, s1, r1, t1 = q2_weights(354, 2 * inner, hidden)
    p2, s2, r2, t2 = q2_weights(355, hidden, inner)
    xb, x = acts(354, m, hidden)
    gate, y0 = rnd(13, hidden).to(DEV), rnd(14, m, hidden).to(DEV)
    h = q2.q2_linear_fused(x, p1, s1, activation="silu", gated=True, out_dtype=torch.bfloat16)
    y = q2.q2_linear_fused(h, p2, s2, gate=gate, residual=y0)
    check(h, O.bf16_to_f64(xb) @ O.unpack_q2(r1, t1).T, "silu", True)
    check(y, host(h) @ O.unpack_q2(r2, t2).T, gate=gate, residual=y0)
