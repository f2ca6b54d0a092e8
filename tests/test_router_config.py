"""The arguments of the scored router that are not tensors as a rule."""
import pytest
import torch

import bit_rotated_weight_b200 as tq


class Logits:
    """A stand-in for CUDA logits, up to the call into the library."""
    is_cuda, dtype, shape, device = True, torch.float32, torch.Size((3, 8)), torch.device("cpu")

    def get_device(self):
        return 0

    def dim(self):
        return 2

    def contiguous(self):
        return self

    def data_ptr(self):
        return 4096


@pytest.fixture
def seen(monkeypatch):
    """(renormalize, scale) of every call that reaches the library."""
    calls = []

    class Library:
        def tq4_1s_router_scored(self, logits, dtype, m, cfg, bias, ids, weights, stream):
            calls.append((cfg.renormalize, cfg.scale))
            return 0

    monkeypatch.setattr(tq, "load_library", Library)
    monkeypatch.setattr(tq, "_current_device", lambda: 0)
    monkeypatch.setattr(tq, "_stream", lambda device: 0)
    return calls


def test_arguments_are_read_on_every_call(seen):
    scale, renorm = torch.tensor(2.5), torch.tensor(True)
    for s, r in ((2.5, True), (0.5, True), (0.5, False), (-1.0, False)):
        scale.fill_(s), renorm.fill_(r)
        tq.tq4_1s_router_scored(Logits(), 2, renormalize=renorm, scale=scale)
    assert seen == [(1, 2.5), (1, 0.5), (0, 0.5), (0, -1.0)]


def test_a_scale_of_zero_has_no_history(seen):
    for s in (-0.0, 0.0):
        tq.tq4_1s_router_scored(Logits(), 2, scale=s)
    assert [str(s) for _, s in seen] == ["0.0", "0.0"]


@pytest.mark.gpu
def test_a_scale_that_changes_in_place():
    z = torch.randn(5, 16, generator=torch.Generator().manual_seed(1)).cuda()
    scale = torch.tensor(2.0)
    _, two = tq.tq4_1s_router_scored(z, 4, scale=scale)
    scale.fill_(4.0)
    _, four = tq.tq4_1s_router_scored(z, 4, scale=scale)
    assert torch.equal(four, 2 * two)
