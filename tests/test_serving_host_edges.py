"""Refusals of the cache's upkeep at its edges (no GPU)."""
import ctypes

import pytest

from gated_deltanet_layer_causal_amd import capi as L

P = ctypes.c_void_p(256)       # never dereferenced: validation fails first
INVALID = 1


@pytest.mark.parametrize("stride", [0, -16])
def test_slots_of_no_bytes_are_refused_before_anything_is_counted(stride):
    """Fork and compact decide in one launch and move in the next, which
    slots of no bytes would leave without a workgroup: the counts would
    change and the call fail."""
    lib = L.load()
    n = lib.gdn_cache_workspace(5)
    assert lib.gdn_cache_fork(P, stride, 5, P, P, 1, P, P, n, None) == INVALID
    assert lib.gdn_cache_compact(P, stride, 5, P, P, P, 1, P, n, None) == INVALID
