"""Rows given with seq_idx that hold one sequence, or hardly more than one (GPU):
their chains cannot be cut into even pieces.  The results are the oracle's, and
the time is that of the row without seq_idx."""
import numpy as np
import pytest
import torch

from tests.test_delta_gpu import check, draw

pytestmark = pytest.mark.gpu

B = torch.bfloat16


def packed(d, starts_of_rows):
    seq = np.zeros(d["v"].shape[:2], np.int32)
    for row, starts in zip(seq, starts_of_rows):
        row[starts] = 1
    return {**d, "seq_idx": torch.from_numpy(np.cumsum(seq, 1).astype(np.int32))}


# heads for which pieces have 16, 32 and 64 columns a CTA, two or three pieces
@pytest.mark.parametrize("H,P,N", [(3, 64, 64), (24, 64, 64), (30, 64, 128), (40, 64, 64),
                                   (30, 128, 64), (60, 64, 128)])
@pytest.mark.parametrize("starts", [[], [5], [64], [590], [130], [300], [200, 410]])
def test_uneven_pieces(H, P, N, starts):
    check(packed(draw(1, 600, H, P, N, 1, B, seed=H, init=True, dfinal=True), [starts]))


@pytest.mark.parametrize("H", [2, 20, 30])
def test_rows_of_both_kinds(H):
    d = draw(2, 530, H, 64, 64, 1, B, seed=H, init=True, dfinal=True)
    check(packed(d, [[], [250, 260]]))
    check(packed(d, [[170, 350], [1]]))


@pytest.mark.parametrize("H,N", [(64, 64), (40, 128), (24, 128)])
def test_one_sequence_takes_no_longer(H, N):
    """Within 12 % of the time without seq_idx (cut without need, the chains of
    64 heads take 30 to 40 % more)."""
    from mamba_selective_state_gb300 import runner
    L = 4096
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda: torch.nn.functional.normalize(r(1, L, 1, N), dim=-1).to(B)  # noqa: E731
    x = [unit(), unit(), r(1, L, H, 64).to(B), (-0.1 * r(1, L, H).abs()).to(B),
         torch.sigmoid(r(1, L, H)).to(B)]
    dy = r(1, L, H, 64).to(B)
    seq = torch.zeros(1, L, dtype=torch.int32, device="cuda")
    devs = [runner.DeltaDevice(*x, dy=dy, seq_idx=s) for s in (None, seq)]

    def time(call):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(10):
            call()
        end.record()
        end.synchronize()
        return start.elapsed_time(end)
    for part in ("fwd", "bwd"):
        calls = [getattr(d, part) for d in devs]
        for c in calls:
            time(c)
        ts = np.array([[time(c) for c in calls] for _ in range(12)]).min(0)
        assert ts[1] <= 1.12 * ts[0], (part, ts)
    assert torch.equal(devs[0].y, devs[1].y) and torch.equal(devs[0].dv, devs[1].dv)
