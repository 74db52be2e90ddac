"""The delta-rule operators together, as the serving example uses them (GPU):
after generation with drafted tokens every sequence's state is the one that
its own tokens give, token by token in 64 bits, from the cached prompt's."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "delta_serving", os.path.join(ROOT, "examples", "delta_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_states_follow_the_kept_tokens():
    ex = example()
    layer = ex.Layer(vocab=64, width=64, nheads=4, headdim=64, dstate=64)
    gen = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, 64, (150,), device="cuda", dtype=torch.int32, generator=gen)
    out, states, kept = ex.generate(layer, prompt, batch=3, new=20, draft=4)
    assert all(len(o) >= 20 and all(0 <= t < 64 for t in o) for o in out)
    assert kept > 0
    # the prompt's state as the sequences got it: bf16 products, then 8 bits
    ins = [t.double().cpu().numpy() for t in layer.inputs(prompt[None, :-1])]
    scale = 64 ** -0.5
    _, start = od.delta_fwd(*ins, scale)
    bits, _ = od.cache_roundtrip(start.astype(np.float32), "int8")
    for i, o in enumerate(out):
        fed = torch.tensor([int(prompt[-1])] + o[:-1], device="cuda", dtype=torch.int32)
        ins = [t.double().cpu().numpy() for t in layer.inputs(fed[None])]
        _, want = od.delta_fwd(*ins, scale, bits.astype(np.float64))
        got = states[i].double().cpu().numpy()
        # the start's error (bf16 products at most 1e-2, and a step of its 8
        # bits where they round the other way, under 1e-2 of the norm) decays
        off = np.linalg.norm(got - want[0]) / np.linalg.norm(want)
        assert off < 2e-2, (i, off)


def test_a_whole_draft_is_kept_when_both_agree():
    ex = example()
    layer = ex.Layer(vocab=64, width=64, nheads=4, headdim=64, dstate=64)
    layer.probs = lambda y, temperature=1.0: ex.Layer.probs(layer, y)   # the draft is the target
    prompt = torch.arange(70, device="cuda", dtype=torch.int32) % 64
    out, _, kept = ex.generate(layer, prompt, batch=2, new=16, draft=3)
    # equal distributions up to the rounding between the steps' token counts:
    # a refusal needs a uniform number within that of 1
    assert kept >= 0.9 * sum(len(o) for o in out) * 3 / 4
