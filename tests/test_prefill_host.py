"""GDNCore.prefill's calls on the host (no GPU): the entry points are replaced
by recorders, so that what each is given can be looked at."""
import contextlib

import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNCore, GDNStateCache

LAUNCHES = ("gdn_cache_copy", "gdn_conv_fwd_state", "gdn_gate_fwd", "gdn_chunk_prepare",
            "gdn_chunk_fwd_states", "gdn_gated_norm_fwd")


@pytest.fixture
def calls(monkeypatch):
    """(name, positional arguments) of every launch, in order."""
    got = []
    for name in LAUNCHES:
        monkeypatch.setattr(L, name, lambda *a, _name=name, **kw: got.append((_name, a)))
    return got


def prefill(core, cache, T, n_seq=2, **other):
    c, bf = core.cfg, torch.bfloat16
    h = torch.zeros(T, c.hv, dtype=bf)
    args = dict(x=torch.zeros(T, c.channels, dtype=bf), w_conv=torch.zeros(c.channels, 4), a=h, b=h,
                A_log=torch.zeros(c.hv), dt_bias=torch.zeros(c.hv), z=torch.zeros(T, c.hv, c.d, dtype=bf),
                w_norm=torch.zeros(c.d), cu_seqlens=torch.tensor([0] + [T] * n_seq, dtype=torch.int32), cache=cache,
                slot_in=torch.arange(n_seq, dtype=torch.int32))
    return core.prefill(**dict(args, **other))


def make():
    core = GDNCore(CoreConfig(1, 2, 32, torch.bfloat16), "cpu")
    return core, GDNStateCache(core.cfg, 4, device="cpu")


def test_every_prefill_has_scratch_of_its_own(calls):
    """Calls on two streams, or one captured and one not, must not share the
    chunk scratch, nor replace each other's."""
    core, cache = make()
    prefill(core, cache, 5)
    prefill(core, cache, 70)
    prefill(core, cache, 5)
    prep = [a[-1] for name, a in calls if name == "gdn_chunk_prepare"]
    states = [a[-1] for name, a in calls if name == "gdn_chunk_fwd_states"]
    assert len(prep) == 3 and all(p is s for p, s in zip(prep, states))
    at = [(w.data_ptr(), w.data_ptr() + w.numel()) for w in prep]     # all alive: kept by `calls`
    assert all(a[1] <= b[0] or b[1] <= a[0] for i, a in enumerate(at) for b in at[:i])
    for T, w in zip((5, 70, 5), prep):
        assert w.numel() >= L.gdn_chunk_fwd_workspace(core.shape(T, 2)) > 0
    assert core._ws is None and core._ws_chunk is None


def test_saved_states_do_not_go_into_scratch():
    core, _ = make()
    z = torch.zeros(1)
    with pytest.raises(ValueError, match="ws_chunk"):
        core.forward(z.view(1, 1), z, z, z, z, z, z, z, torch.zeros(2, dtype=torch.int32), ws_chunk=z)


def test_prefill_runs_on_the_caches_device(calls, monkeypatch):
    """The copies from and into the cache and the chunked forward go to one
    device's stream, whichever device is the current one."""
    core, cache = make()
    on = []

    @contextlib.contextmanager
    def current(dev):
        on.append((dev, len(calls)))
        yield
        on.append((dev, len(calls)))

    monkeypatch.setattr(L, "current_device", current, raising=False)
    prefill(core, cache, 5)
    assert on == [(cache.buffer.device, 0), (cache.buffer.device, len(calls))] and len(calls) == 9


def test_prefill_refuses_tensors_on_other_devices(calls):
    core, cache = make()
    for name in ("x", "w_conv", "a", "b", "A_log", "dt_bias", "z", "w_norm", "cu_seqlens", "slot_in", "slot_out"):
        t = torch.zeros(5, 128, dtype=torch.bfloat16) if name == "x" else torch.zeros(3 if name == "cu_seqlens" else 2)
        with pytest.raises(ValueError, match=f"{name} is on meta, the cache on cpu"):
            prefill(core, cache, 5, **{name: t.to("meta")})
    assert not calls


def test_prefill_of_no_tokens_passes_states_through(calls, monkeypatch):
    """A batch of empty sequences: what step() does with one."""
    core, cache = make()
    monkeypatch.setattr(L, "gdn_step_fwd", lambda *a, **kw: calls.append(("gdn_step_fwd", a)))
    out = prefill(core, cache, 0, slot_out=torch.tensor([2, 3], dtype=torch.int32))
    assert [name for name, _ in calls] == ["gdn_step_fwd"] and out.shape == (0, 2, 32)
    slot_in, slot_out = calls[0][1][11:13]
    assert slot_in.tolist() == [0, 1] and slot_out.tolist() == [2, 3]
