"""The counters of attention that is split along the keys: captures on streams that no eager call
has used, and graphs that were replayed at once, spoil no other call."""
import numpy as np
import pytest

import gguf_q4_dequant_amd as q4k
from tests.gpu_helpers import fresh_stream, to_dev
from tests.layer_reference import Paged, rng_of

pytestmark = pytest.mark.gpu


def batch(tag, sizes):
    rng = rng_of(100, tag)
    p = Paged(rng, sizes, 2, 64, 16, "f16")
    cache, seqs = p.on_device()
    return to_dev(rng.standard_normal((p.T, 8, 64)).astype(np.float32)), cache, seqs


def captured(stream, calls, mode="global"):
    import torch
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(g, stream=stream, capture_error_mode=mode):
            outs = [q4k.attention(*c) for c in calls]
    return g, outs


def test_a_capture_needs_an_eager_call_first():
    """Without one the words that count would not be zeroed before the stream's eager calls: refused."""
    import torch
    call = batch(0, [(900, 1), (40, 1)])
    want = q4k.attention(*call)
    side = fresh_stream()
    torch.cuda.synchronize()
    x = torch.ones(8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side, capture_error_mode="relaxed"):
            x += 1
            with pytest.raises(q4k.Q4KError):
                q4k.attention(*call)
        assert torch.equal(q4k.attention(*call), want)
        side.synchronize()
    g, outs = captured(side, [call, call], "relaxed")
    for _ in range(3):
        [o.fill_(float("nan")) for o in outs]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_replays_at_once_spoil_only_themselves():
    """Two graphs captured on one stream share its workspace and are not to run at once: what they give
    then is not looked at; afterwards each of them, eager calls and a graph captured later are right."""
    import torch
    calls = [batch(1, [(2000, 1), (50, 1)]), batch(2, [(700, 3), (900, 2), (10, 1)]), batch(3, [(3000, 1)])]
    want = [q4k.attention(*c) for c in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            q4k.attention(*c)
        side.synchronize()
    graphs = [captured(side, calls), captured(side, calls[::-1] + calls[:1])]
    wants = [want, want[::-1] + want[:1]]
    others = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for rep in range(6):
        for _ in range(20):
            for (g, _), stream in zip(graphs, others):
                with torch.cuda.stream(stream):
                    g.replay()
        with torch.cuda.stream(side):  # and eager calls at the same time
            eager = [q4k.attention(*c) for c in calls for _ in range(5)]
        torch.cuda.synchronize()
        del eager
        for (g, outs), expected in list(zip(graphs, wants))[::1 if rep % 2 else -1]:
            [o.fill_(float("nan")) for o in outs]
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, expected))
        with torch.cuda.stream(side):
            got = [q4k.attention(*c) for c in calls]
            side.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(got, want))
    g, outs = captured(side, calls)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_eager_calls_and_replays_in_turn():
    """Calls take their counters in turn: any order of eager calls, of graphs of one and of several calls."""
    import torch
    calls = [batch(4, [(1500, 1), (50, 1)]), batch(5, [(600, 2), (800, 1)]), batch(6, [(2500, 1)])]
    want = [q4k.attention(*c) for c in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            q4k.attention(*c)
        side.synchronize()
    graphs = [(captured(side, [calls[i] for i in which]), which) for which in ((0,), (1, 2), (0, 1, 2), (2,))]
    rng = rng_of(101)
    with torch.cuda.stream(side):
        for _ in range(40):
            if rng.random() < 0.5:
                i = int(rng.integers(3))
                assert torch.equal(q4k.attention(*calls[i]), want[i])
            else:
                (g, outs), which = graphs[int(rng.integers(4))]
                [o.zero_() for o in outs]
                g.replay()
                assert all(torch.equal(o, want[i]) for o, i in zip(outs, which))
