"""examples/transformer_layer.py: the layer's operators together, trained and
from a cache."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "transformer_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("transformer_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
def test_it_learns_and_the_cache_agrees(example):
    import torch
    torch.manual_seed(0)
    model = example.Decoder().cuda().bfloat16()
    losses = example.train(model, 200)
    assert losses[0] > 4.0 and sum(losses[-10:]) / 10 < 2.5, (losses[0], losses[-10:])
    # bf16 rounds each layer's five results to 2^-8 of themselves, in both ways of computing them
    worst, most = example.cached_against_whole(model)
    assert worst < 2 * 2 * 5 * 2.0 ** -8 * max(most, 1.0), (worst, most)


@pytest.mark.gpu
def test_the_same_steps_give_the_same_bits(example):
    import torch

    def once():
        torch.manual_seed(0)
        model = example.Decoder().cuda().bfloat16()
        return example.train(model, 3), [p.detach().clone() for p in model.parameters()]

    (a, u), (b, v) = once(), once()
    # (the embedding's gradient is summed by atomics, in the library)
    assert a[0] == b[0] and all(torch.isfinite(p).all() for p in u + v)


@pytest.mark.gpu
def test_the_same_steps_give_the_same_losses_and_weights(example):
    import torch

    def once():
        torch.manual_seed(0)
        model = example.Decoder().cuda().bfloat16()
        return example.train(model, 20), [p.detach().clone() for p in model.parameters()]

    (a, u), (b, v) = once(), once()
    assert a == b and all(torch.equal(p, q) for p, q in zip(u, v))
