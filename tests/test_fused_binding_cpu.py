"""The binding of the fused and grouped linears, the router and the combination, without a GPU: what it hands to the
library when an input without elements, which no kernel reads, is a host tensor."""
import types

import pytest
import torch

import ternary_weight_quantized_q2_amd as q2


class Recorder:
    """Stands for the library: entry points succeed and note that they were called, sizes are 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 0
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(q2, "load", lambda: rec)
    monkeypatch.setattr(q2, "_here", lambda: 0)
    monkeypatch.setattr(q2, "_stream", lambda: 0)
    made = []
    # allocations on the device are noted, and made on the host here
    monkeypatch.setattr(q2, "torch", types.SimpleNamespace(**{n: getattr(torch, n) for n in dir(torch) if n[0] != "_"}))

    def empty(shape, dtype=None, device=None):
        made.append(str(device))
        return torch.empty(shape, dtype=dtype)

    monkeypatch.setattr(q2.torch, "empty", empty)
    rec.made = made
    return rec


bf, u8, f16, i32 = torch.bfloat16, torch.uint8, torch.float16, torch.int32


def test_output_of_an_empty_sum_is_on_the_device(lib):
    q2.q2_linear_fused(torch.empty((4, 0), dtype=bf), torch.empty((6, 0), dtype=u8), torch.empty((6, 0), dtype=f16))
    assert lib.calls == ["q2_linear_fused"] and lib.made == ["cuda:0"]


def test_output_of_empty_4bit_sum_is_on_the_device(lib):
    e = torch.empty((6, 0), dtype=f16)
    q2.q4_linear_fused(torch.empty((4, 0), dtype=bf), torch.empty((6, 0), dtype=u8), e, e)
    assert lib.calls == ["q4_linear_fused"] and lib.made == ["cuda:0"]


def test_route_of_no_tokens_is_on_the_device(lib):
    q2.q2_route(torch.empty((0, 5)), 2)
    assert lib.calls == ["q2_route"] and lib.made == ["cuda:0"] * 4      # the fifth is made like the first


def test_combination_of_no_rows_is_on_the_device(lib):
    q2.q2_combine(torch.empty((0, 8)), torch.empty((3, 0), dtype=i32), torch.empty((3, 0)))
    assert lib.calls == ["q2_combine"] and lib.made == ["cuda:0"]
