"""Copies of a state cache: deep ones, pickled ones and saved ones have
memory of their own, which their calls read and write."""
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNStateCache
from tests.test_block_copies import COPIES

DEV = "cuda:0"
CFG = CoreConfig(hk=1, hv=2, d=32)


@pytest.mark.parametrize("seen", [False, True])
@pytest.mark.parametrize("how", COPIES)
def test_a_copy_names_its_own_memory(how, seen):
    """seen: its layers' views were asked for before the copy."""
    cache = GDNStateCache(CFG, 4, 2, device="cpu")
    cache.buffer.fill_(7)
    if seen:
        cache.S(0), cache.conv(1)
    c = COPIES[how](cache)
    s = c._slots
    assert s.ptrs == (c.buffer.data_ptr(), c.refs.data_ptr(), s.ws.data_ptr(), s.ws.numel())
    assert not set(s.ptrs[:3]) & set(cache._slots.ptrs[:3])
    assert (s.device, s.index) == (c.buffer.device, -1)
    assert c.layer(1).S_ptr == c.S(1).data_ptr() == c.buffer.data_ptr() + c.slot_bytes // 2
    assert torch.equal(c.buffer, cache.buffer)
    c.buffer.zero_()
    assert (cache.buffer == 7).all() and (c.conv(1) == 0).all() and (c.S(0) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES)
def test_a_copy_goes_on_alone(how):
    """Slots taken, counted, released and moved in a copy leave the original
    as it is, and the other way round."""
    cache = GDNStateCache(CFG, 4)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    slots = cache.fork(ints(-1, -1))
    assert slots.tolist() == [0, 1]
    cache.S().normal_()
    c = COPIES[how](cache)
    states, refs = cache.S().clone(), cache.refs.clone()
    assert torch.equal(c.S(), states) and torch.equal(c.refs, refs)
    taken = c.fork(slots)
    assert taken.tolist() == [2, 3] and torch.equal(c.S()[2:], states[:2])
    c.retain(ints(0))
    c.release(ints(1))
    table = taken.clone()
    assert c.compact(table).tolist() == [0, -1, 2, 1] and table.tolist() == [2, 1]     # only the last one moves
    assert c.refs.tolist() == [2, 1, 1, 0] and torch.equal(c.S()[:3], states[[0, 1, 0]])
    assert torch.equal(cache.S(), states) and torch.equal(cache.refs, refs)
    cache.release(slots)
    assert cache.refs.tolist() == [0] * 4 and c.refs.tolist() == [2, 1, 1, 0]


def test_the_views_of_the_c_abi_refuse_to_be_copied():
    """A layer's view names memory that a copy of it would not own."""
    view = GDNStateCache(CFG, 4, device="cpu").layer()
    assert isinstance(view, L.Cache)
    for how in ("deepcopy", "pickle"):
        with pytest.raises(ValueError):
            COPIES[how](view)
