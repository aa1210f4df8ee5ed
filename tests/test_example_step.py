"""examples/zero_step.py: the whole sharded step trains, with either state
width, and repeats itself."""
import importlib.util
import math
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("zero_step", os.path.join(ROOT, "examples", "zero_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_the_sharded_step_trains(bits):
    losses = load().train(steps=60, state_bits=bits)
    assert abs(losses[0] - math.log(500)) < 0.1            # near-uniform logits at the start
    assert losses[-1] < 2.0                                # the data's own entropy is ln 3 = 1.10
    assert all(math.isfinite(x) for x in losses)


@pytest.mark.gpu
def test_the_sharded_step_repeats():
    m = load()
    a, b = m.train(steps=4, state_bits=8), m.train(steps=4, state_bits=8)
    assert a == b
