"""The calls that write states in place, on streams other than the current one: what
they do to the states, beside what they return."""
import pytest

torch = pytest.importorskip("torch")

import sparse_weight_direct_gb300 as swd  # noqa: E402
from test_sequence import Draw  # noqa: E402
from test_sequence_edges import busy  # noqa: E402


def step_and_reorder():
    """Of each: the states it is given, and the call."""
    d = Draw(21)
    x, r, A = d(8, 300), d(8, 300), -d(300).abs()
    slots = torch.tensor([3, 8, 0, 5, 1, 7, 2, 6], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[0, 0, 2, 2], [3, 3, 3, 1]], dtype=torch.int32, device="cuda")
    return {
        "gated_scan_step": (d(9, 300), lambda pool, s: swd.gated_scan_step(pool, x, r, A, slots=slots, stream=s)),
        "reorder_states": (d(9, 70000), lambda pool, s: swd.reorder_states([pool], parents, slots.view(2, 4), stream=s)),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["gated_scan_step", "reorder_states"])
def test_states_on_another_stream(name, raw):
    """The states as a call on the current stream leaves them, while that stream is busy."""
    states, call = step_and_reorder()[name]
    after = states.clone()
    want = call(after, None).clone()
    pool, work, side = states.clone(), busy(), torch.cuda.Stream()
    torch.cuda.synchronize()
    work()
    end = torch.cuda.Event()
    end.record()
    got = call(pool, side.cuda_stream if raw else side)
    early = not end.query()
    torch.cuda.synchronize()
    assert early, "the queue was too short to show anything"
    assert torch.equal(got, want) and torch.equal(pool, after) and not torch.equal(pool, states)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gated_scan_step", "reorder_states"])
def test_states_of_two_streams_at_once(name):
    """Two streams through the same call side by side, each with states of its own."""
    states, call = step_and_reorder()[name]
    after = states.clone()
    want = call(after, None).clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pools = [[states.clone() for _ in streams] for _ in range(4)]
    torch.cuda.synchronize()
    got = [[call(p, s) for p, s in zip(row, streams)] for row in pools]
    torch.cuda.synchronize()
    for row, out in zip(pools, got):
        for p, o in zip(row, out):
            assert torch.equal(o, want) and torch.equal(p, after)
