"""int8 products are whole numbers as long as their partial sums stay below 2^24,
however near to it they come (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# each way that a product can go; 1024 codes of -128 sum up to 2^24 itself
@pytest.mark.parametrize("m,n", [(1, 300), (20, 300), (100, 500), (300, 1000), (9000, 1100)])
@pytest.mark.parametrize("k,lo,hi", [(1024, 100, 128), (1024, -128, -100), (1023, 120, 128), (700, -128, 128), (1024, -128, -127)])
def test_sums_near_two_to_the_24(m, n, k, lo, hi):
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(m + k)
    a, w = (torch.randint(lo, hi, (r, k), generator=g, device="cuda").to(torch.int8) for r in (m, n))
    out = runner.Linear8(w, torch.ones(n, device="cuda"), out_dtype=torch.float32)(a, torch.ones(m, device="cuda"))
    assert torch.equal(out.double(), a.double() @ w.double().T)
