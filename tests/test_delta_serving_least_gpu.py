"""The serving example at its smallest arguments (GPU): no drafted tokens, and a
prompt of one token."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from tests.test_delta_serving_gpu import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,draft", [(1, 0), (1, 2), (70, 0)])
def test_smallest_arguments(prompt, draft):
    ex = example()
    layer = ex.Layer(vocab=64, width=64, nheads=2, headdim=64, dstate=64, ngroups=1)
    prompt = torch.arange(prompt, device="cuda", dtype=torch.int32) % 64
    out, states, kept = ex.generate(layer, prompt, batch=2, new=6, draft=draft)
    assert all(len(o) >= 6 and all(0 <= t < 64 for t in o) for o in out)
    assert draft or (kept == 0 and all(len(o) == 6 for o in out))
    if len(prompt) > 1:
        return
    # from an empty state every sequence's is the one that its own tokens give, in fp32
    for i, o in enumerate(out):
        fed = torch.tensor([int(prompt[-1])] + o[:-1], device="cuda", dtype=torch.int32)
        ins = [t.double().cpu().numpy() for t in layer.inputs(fed[None])]
        _, want = od.delta_fwd(*ins, 64 ** -0.5)
        got = states[i].double().cpu().numpy()
        # products whose inputs a GEMM of another shape may round the other way to bf16
        assert np.linalg.norm(got - want[0]) < 1e-2 * np.linalg.norm(want)
