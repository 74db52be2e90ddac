"""The status words of one Linear8's calls (GPU): calls that may overlap, on
different streams or in different graphs, do not clear one another's."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def maps(m, k=256):
    """A map, its weights, and m tokens; k = 256 needs no memory but the status word."""
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(m)
    code = lambda r: torch.randint(-60, 61, (r, k), generator=g, device="cuda").to(torch.int8)  # noqa: E731
    return (runner.Linear8(code(300), torch.rand(300, generator=g, device="cuda")), code(m),
            torch.rand(m, generator=g, device="cuda"))


def expire(word):
    """As a bounded wait that ran out leaves it."""
    word[:4].view(torch.int32).fill_(1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("m", [3, 100])
def test_calls_on_other_streams_leave_it(m):
    from mamba_selective_state_gb300 import _lib
    lin, a, s = maps(m)
    torch.cuda.synchronize()
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    words = []
    for st in streams:
        lin(a, s, stream=st)
        words.append(lin.workspace)
    assert len({w.data_ptr() for w in words}) == 3
    torch.cuda.synchronize()
    expire(words[0])
    for st in streams[1:]:
        lin(a, s, stream=st)
    assert lin.device_status() == _lib.SSD_OK
    assert _lib.ssd_read_device_status(words[0]) == _lib.SSD_ERR_TIMEOUT
    lin(a, s)                                   # the same stream's next call clears it
    assert lin.device_status() == _lib.SSD_OK and _lib.ssd_read_device_status(words[0]) == _lib.SSD_OK


@pytest.mark.parametrize("m", [3, 100])
def test_graphs_have_their_own(m):
    from mamba_selective_state_gb300 import _lib
    lin, a, s = maps(m)
    want = lin(a, s).clone()
    eager = lin.workspace
    graphs, outs, words = [], [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(lin(a, s))
            words.append(lin.workspace)
            outs.append(lin(a, s))
            words.append(lin.workspace)
    assert len({w.data_ptr() for w in words + [eager]}) == 5
    for w in words + [eager]:
        expire(w)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert [_lib.ssd_read_device_status(w) for w in words + [eager]] == [_lib.SSD_OK] * 2 + [_lib.SSD_ERR_TIMEOUT] * 3
    graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert _lib.ssd_read_device_status(eager) == _lib.SSD_ERR_TIMEOUT


def test_the_last_call_is_waited_for_wherever_it_ran():
    """The status is read behind the last call, also where that was given a stream
    and none is named here: the word that is found holds what the call left."""
    from mamba_selective_state_gb300 import _lib
    lin, a, s = maps(9000)                      # (needs more memory than the word)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lin(a, s, stream=side)
    word = lin.workspace[:4].view(torch.int32)
    for value, n in ((0, 1), (1, 20)):          # (once before, so that every kernel is loaded)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            wait = torch.randn(6000, 6000, device="cuda")
            for _ in range(n):                  # some milliseconds of work ahead of the word's writer
                wait = wait @ wait
                wait = wait / wait.abs().max()
            word.fill_(value)
    assert lin.device_status() == _lib.SSD_ERR_TIMEOUT
