"""Draft verification where several CTAs share a sequence's words (GPU): drafts
without probabilities, the fallback to the target's row, ties and empty rows, with
1, 2, 4 and 8 CTAs.  Whole numbers: they are equal."""
import pytest
import torch

from tests.test_serving_gpu import draft_case, verify

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16

# words for 1, 2, 4 and 8 CTAs of a few sequences; a last CTA with a few words less
WORDS = [2048, 2049, 4095, 4097, 8192, 8193, 20001, 32768, 100003]


@pytest.mark.parametrize("V", WORDS)
@pytest.mark.parametrize("dtype", [F, B])
def test_drafts_without_probabilities(V, dtype):
    """The refused token weighs one less than the target gives it: nothing."""
    c = draft_case(6, 3, V, dtype, seed=V)
    c["draft"] = None
    for i, x in enumerate((0, V - 1, V // 2, V // 8, V // 8 - 1, 7)):  # at the CTAs' edges too
        c["tokens"][i, 0] = x
        c["uniform"][i, 0] = 2.0                       # refused
        c["noise"][i, x] = 1e-20                       # it would win the race
    tokens, kept = verify(c)
    assert not kept.any()
    assert all(tokens[i, 0] != c["tokens"][i, 0] for i in range(6))


@pytest.mark.parametrize("V", WORDS)
def test_kept_and_refused_drafts_without_probabilities(V):
    c = draft_case(5, 4, V, F, seed=V + 1, ragged=True)
    c["draft"] = None
    c["uniform"][:] = torch.tensor([[0.0, 2.0, 0.0, 0.0]] * 5)
    verify(c)


@pytest.mark.parametrize("V", WORDS)
@pytest.mark.parametrize("dtype", [F, B])
def test_fallback_and_empty_rows(V, dtype):
    c = draft_case(7, 2, V, dtype, seed=V + 2)
    c["uniform"][:, 0] = 2.0                           # all refused
    c["draft"][:3, 0] = c["target"][:3, 0]             # nothing left of w: the target's row
    c["target"][3, 0], c["draft"][3, 0] = 0.0, 0.0     # nor of that: token 0
    c["target"][4, 0] = float("nan")
    c["draft"][5, 0] = c["target"][5, 0]
    c["noise"][5] = 1.0
    c["target"][5, 0] = c["draft"][5, 0] = 0.5         # every word ties: the lowest
    c["draft"][6, 0] = c["target"][6, 0]
    c["target"][6, 0, V - 1] += 0.25                   # one word left, the last CTA's last
    tokens, kept = verify(c)
    assert not kept.any()
    assert tokens[3, 0] == 0 and tokens[4, 0] == 0 and tokens[5, 0] == 0 and tokens[6, 0] == V - 1


@pytest.mark.parametrize("b", [1, 40, 80, 160, 400])
def test_batches_with_fewer_ctas_a_sequence(b):
    verify(draft_case(b, 2, 9000, B, seed=b, ragged=True))
    c = draft_case(b, 1, 9000, F, seed=b + 1)
    c["draft"] = None
    verify(c)
