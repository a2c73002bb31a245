"""Outputs of the sampler that overlap what it reads, refused before any HIP call, and the sizes from which it cuts rows:
no GPU is needed."""
import ctypes

import pytest

import ternary_weight_quantized_q2_amd as q2

FAKE = 1 << 20          # 256-byte aligned fake device addresses (never dereferenced)
B, V = 4, 100
OUT = 4 * B             # bytes of an output


@pytest.fixture(scope="module")
def lib():
    return q2.load()


def sample(lib, ld=V, flags=0, b=B, v=V, logits=FAKE, u=FAKE << 1, token=FAKE << 2, prob=FAKE << 3, **rows):
    s = q2.Sampling(1.0, 0, 1.0, 0.0, *(rows.get(n) for n in ("temperature", "top_k", "top_p", "min_p")))
    st = lib.q2_sample(logits, b, v, ld, flags, ctypes.addressof(s), u, token, prob, FAKE << 4, 1 << 40, None)
    return st, lib.q2_last_error().decode()


def refused(got, text):
    return got[0] == q2.Q2_ERR_ARG and text in got[1]


def passes(lib, **kw):
    """No output overlaps anything but what is checked last, which is made to overlap: nothing is launched."""
    return refused(sample(lib, **{**kw, "min_p": kw.get("prob", FAKE << 3)}), "prob overlaps min_p")


@pytest.mark.parametrize("name", ["token", "prob"])
def test_outputs_over_logits(lib, name):
    for flags, size in ((0, 4), (q2.Q2_SAMPLE_LOGITS_BF16, 2)):
        end = FAKE + B * V * size
        for at in (FAKE, FAKE + 40, end - 4, FAKE - OUT + 4):
            assert refused(sample(lib, flags=flags, **{name: at}), f"{name} overlaps the logits"), at
        for at in (end, FAKE - OUT):
            assert passes(lib, flags=flags, **{name: at}), at


@pytest.mark.parametrize("name", ["token", "prob"])
def test_outputs_between_rows_of_logits(lib, name):
    """Rows of 400 bytes, 416 apart: an output of 16 fits between two."""
    for row in range(B - 1):
        gap = FAKE + 416 * row + 400
        assert passes(lib, ld=104, **{name: gap})
        for at in (gap - 4, gap + 4, FAKE + 416 * (row + 1) + 200):
            assert refused(sample(lib, ld=104, **{name: at}), "logits"), at
    assert passes(lib, ld=104, **{name: FAKE + 416 * (B - 1) + 400})
    assert passes(lib, ld=1, b=1, **{name: FAKE + 400}) and refused(sample(lib, ld=1, b=1, **{name: FAKE + 396}), "logits")


def test_outputs_over_each_other(lib):
    for at in (0, 4, OUT - 4, -4, 4 - OUT):
        assert refused(sample(lib, token=FAKE << 2, prob=(FAKE << 2) + at), "token overlaps prob"), at
    for at in (OUT, -OUT):
        assert passes(lib, token=FAKE << 2, prob=(FAKE << 2) + at), at


@pytest.mark.parametrize("name", ["token", "prob"])
def test_outputs_over_u_and_settings(lib, name):
    out = FAKE << (2 if name == "token" else 3)
    for at in (4, OUT - 4, -4, 4 - OUT):
        assert refused(sample(lib, u=out + at), f"{name} overlaps u"), at
        for rows in ("temperature", "top_k", "top_p", "min_p"):
            assert refused(sample(lib, **{rows: out + at}), f"{name} overlaps {rows}"), (rows, at)
    for at in (0, OUT, -OUT):
        assert passes(lib, u=out + at), at
    for rows in ("temperature", "top_k", "top_p", "min_p"):
        assert refused(sample(lib, **{rows: out}), f"{name} overlaps {rows}"), rows
    for rows in ("temperature", "top_k", "top_p"):
        assert passes(lib, **{rows: out + OUT}) and passes(lib, **{rows: out - OUT})


def test_empty_outputs_overlap_nothing(lib):
    assert sample(lib, b=0, token=FAKE, prob=FAKE, u=FAKE)[0] == q2.Q2_OK


@pytest.mark.parametrize("b,v,cut", [(1, 16384, False), (1, 20000, True), (8, 18000, False), (8, 24000, True), (16, 20000, False),
                                     (16, 24000, True), (32, 24000, False), (32, 40000, True), (48, 28000, False), (64, 32768, False),
                                     (64, 50021, True), (80, 36000, False), (96, 40000, False), (96, 64000, True),
                                     (128, 50021, False), (128, 128009, True), (129, 1 << 24, False)])
def test_rows_are_cut_where_that_measured_less(b, v, cut):
    """A workspace is needed where several workgroups share a row."""
    assert (q2.sample_workspace_bytes(b, v) > 0) == cut
