"""How the documentation has random numbers advance: no mask is drawn twice (CPU only)."""
import os
import re

import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def advances():
    """Every statement in the examples that advances rng."""
    text = open(os.path.join(ROOT, "README.md")).read() + coat.dropout.__doc__
    return re.findall(r"\brng(?:\[\w+\])? \+= \w+", text)


def draws(statement, ranks=4, layers=3, steps=5):
    """(key, counter) of every layer's mask on every rank, seeds one apart."""
    for rank in range(ranks):
        rng = torch.tensor([1000 + rank, 0])
        for _ in range(steps):
            for offset in range(layers):
                yield int(rng[0]), int(rng[1]) + offset
            exec(statement, dict(rng=rng, layers=layers, n=layers))


def test_no_mask_is_drawn_twice():
    found = advances()
    assert len(found) >= 2
    for statement in found:
        all_of = list(draws(statement))
        assert len(set(all_of)) == len(all_of) == 60, statement


def test_seed_and_step_together_would_repeat():
    """Rank r's mask of a layer is rank r + 1's of the next layer a step earlier."""
    all_of = list(draws("rng += 1"))
    assert len(set(all_of)) < len(all_of)
    a = ref.factors(4, 24, 0.5, torch.tensor([1000 + 1, 0 + 1]), 0)   # rank 0 after one step
    b = ref.factors(4, 24, 0.5, torch.tensor([1000 + 1, 0]), 1)       # rank 1 before it, next layer
    assert torch.equal(a, b)
