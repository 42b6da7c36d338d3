"""GDNCore.prefill on the GPU: several at once, captured, and at its edges.
Values are compared with the same calls made one after the other, bit by bit
(the chunked form's own accuracy is tested with its entry points)."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_causal_amd.layer import GDNStateCache
from tests.gpu_util import host
from tests.test_gpu_serving import Case, ints

pytestmark = pytest.mark.gpu


def test_two_caches_of_one_core_on_two_streams():
    """Order is asked for per cache only: the calls share no scratch."""
    cs = [Case("bf16", 4, 8, 128, [700, 300, 64, 1, 500], 5, seed=s) for s in (1, 2)]
    core, slots = cs[0].core, ints([4, 2, 0, 1, 3])
    args = [c.args() for c in cs]
    start = [c.cache.buffer.clone() for c in cs]
    want = [(core.prefill(*args[i], c.cache, slots).clone(), c.cache.buffer.clone()) for i, c in enumerate(cs)]
    streams = [torch.cuda.Stream() for _ in cs]
    for k in range(5):
        for c, s in zip(cs, start):
            c.cache.buffer.copy_(s)
        torch.cuda.synchronize()
        got = [None, None]
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i] = core.prefill(*args[i], c.cache, slots)
        torch.cuda.synchronize()
        for i, c in enumerate(cs):
            assert torch.equal(got[i], want[i][0]) and torch.equal(c.cache.buffer, want[i][1]), (k, i)


def test_captured_and_replayed_beside_longer_calls():
    """A captured prefill keeps its scratch: a longer eager one in between
    neither takes it nor is changed by the replays."""
    c = Case("bf16", 2, 4, 128, [90, 3], 3, seed=5)
    long = Case("bf16", 2, 4, 128, [900, 40], 3, seed=6)
    core, slots = c.core, ints([2, 0])
    args, largs = c.args(), long.args()
    other = GDNStateCache(core.cfg, 3, device="cuda")
    other.buffer.copy_(long.cache.buffer)
    start, lstart = c.cache.buffer.clone(), other.buffer.clone()
    want = core.prefill(*args, c.cache, slots).clone()
    after = c.cache.buffer.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        core.prefill(*args, c.cache, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = core.prefill(*args, c.cache, slots)
    lwant = lafter = None
    for k in range(4):
        other.buffer.copy_(lstart)
        lgot = core.prefill(*largs, other, slots)
        torch.cuda.synchronize()
        if lwant is None:
            lwant, lafter = lgot.clone(), other.buffer.clone()
        assert torch.equal(lgot, lwant) and torch.equal(other.buffer, lafter), k
        c.cache.buffer.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.cache.buffer, after), k
        assert torch.equal(lgot, lwant) and torch.equal(other.buffer, lafter), k


def test_no_tokens_pass_states_through():
    c = Case("bf16", 1, 2, 128, [0, 0, 0], 6)
    got = c.core.prefill(*c.args(), c.cache, ints([0, 3, -1]), ints([1, 3, 4]))
    assert got.shape == (0, 2, 128)
    S, conv = c.S.copy(), c.conv.copy()
    S[1], conv[1], S[4], conv[4] = S[0], conv[0], 0, 0
    assert np.array_equal(host(c.cache.S()), S) and np.array_equal(host(c.cache.conv()), conv)
