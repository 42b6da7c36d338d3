"""A cache of Gated DeltaNet states for serving: one buffer of slots, each
holding all layers' states of one sequence, with its upkeep on the device.

Slot layout, layer after layer (each padded to 256 bytes): the fp32 state
[hv, d, d], then the last three conv input rows [3, C] in the storage type.
Layers of a slot lie together, so that taking, copying or moving a sequence
is one contiguous copy.
"""
from __future__ import annotations

import torch

from . import capi as L


class GDNStateCache:
    """n_slots slots for n_layers layers of one CoreConfig.

    refs [n_slots] (int32, device) counts the users of each slot; a slot with
    count 0 is free.  Slots are named by int32 device tensors, and every call
    is asynchronous on the current stream: nothing here waits for the device.
    Calls on one cache must be ordered (one stream, or events between)."""

    ALIGN = 256

    def __init__(self, cfg, n_slots: int, n_layers: int = 1, device="cuda", buffer=None, refs=None):
        """buffer (uint8 [n_slots, slot_bytes], contiguous) and refs (int32
        [n_slots]): memory to use instead of new memory, taken as it is."""
        if n_slots < 1 or n_layers < 1:
            raise ValueError("a cache needs at least one slot and one layer")
        C, E = cfg.channels, cfg.dtype.itemsize
        self.cfg, self.n_slots, self.n_layers = cfg, n_slots, n_layers
        s_bytes, c_bytes = cfg.hv * cfg.d * cfg.d * 4, 3 * C * E
        layer = (s_bytes + c_bytes + self.ALIGN - 1) // self.ALIGN * self.ALIGN
        self.slot_bytes = n_layers * layer
        dev = torch.device(device)
        if buffer is None:
            buffer = torch.empty((n_slots, self.slot_bytes), dtype=torch.uint8, device=dev)
        elif buffer.dtype != torch.uint8 or tuple(buffer.shape) != (n_slots, self.slot_bytes) or \
                not buffer.is_contiguous():
            raise ValueError(f"buffer must be a contiguous uint8 [{n_slots}, {self.slot_bytes}] tensor")
        if refs is None:
            refs = torch.zeros(n_slots, dtype=torch.int32, device=buffer.device)
        elif refs.dtype != torch.int32 or tuple(refs.shape) != (n_slots,) or \
                refs.device != buffer.device or not refs.is_contiguous():
            raise ValueError(f"refs must be a contiguous int32 [{n_slots}] tensor on the buffer's device")
        self._layer_bytes, self._parts = layer, (s_bytes, c_bytes)
        self._dims = cfg.hv, cfg.d, C, cfg.dtype
        self._layers = [None] * n_layers     # views, made when first asked for
        self._slots = L.Slots(buffer, refs, torch.empty(L.gdn_cache_workspace(n_slots),
                                                        dtype=torch.uint8, device=buffer.device))

    @property
    def buffer(self) -> torch.Tensor:
        """All slots, uint8 [n_slots, slot_bytes]."""
        return self._slots.buf

    @property
    def refs(self) -> torch.Tensor:
        """The users of each slot, int32 [n_slots]."""
        return self._slots.refs

    def layer(self, k: int = 0) -> L.Cache:
        """The C ABI's view of layer k."""
        got = self._layers[k]
        if got is None:
            (hv, d, C, dtype), buf = self._dims, self.buffer
            at = k % self.n_layers * self._layer_bytes
            mid, end = at + self._parts[0], at + sum(self._parts)
            S = buf[:, at:mid].view(torch.float32).view(self.n_slots, hv, d, d)
            conv = buf[:, mid:end].view(dtype).view(self.n_slots, 3, C)
            got = self._layers[k] = L.make_cache(S, conv)
        return got

    def S(self, k: int = 0) -> torch.Tensor:
        """Layer k's states [n_slots, hv, d, d], a view."""
        return self.layer(k).S

    def conv(self, k: int = 0) -> torch.Tensor:
        """Layer k's conv rows [n_slots, 3, C], a view."""
        return self.layer(k).conv

    def fork(self, src: torch.Tensor) -> torch.Tensor:
        """Takes a free slot for every request: filled with a copy of slot
        src[i], or with zeros where src[i] is -1 (a new sequence).  Returns
        the slots (int32); -1 where the request could not be served (no free
        slot left, or src[i] is no live slot) or src[i] < -1 (no request)."""
        dst = torch.empty_like(src)
        self._slots.fork(src, dst)
        return dst

    def retain(self, slots: torch.Tensor) -> None:
        """One more user of each live slot named."""
        self._slots.count("gdn_cache_retain", slots)

    def release(self, slots: torch.Tensor) -> None:
        """One user less of each slot named; at 0 the slot is free."""
        self._slots.count("gdn_cache_release", slots)

    def copy(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Slot dst[i] = slot src[i] (zeros where src[i] < 0), counts left alone."""
        L.gdn_cache_copy(self.buffer, self.buffer, src, dst)

    def compact(self, table: torch.Tensor | None = None) -> torch.Tensor:
        """Moves the live slots to the front of the cache.  Returns each
        slot's new place (int32 [n_slots], -1 for free ones) and rewrites
        `table` (int32, any length: the slots of the running sequences) by it."""
        remap = torch.empty_like(self.refs)
        self._slots.compact(remap, table)
        return remap
