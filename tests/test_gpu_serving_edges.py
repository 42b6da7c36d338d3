"""The recurrent form over cached states on the GPU, at the edges of its
launches: the most sequences and heads that a call takes, thousands of groups
at d = 128, and slots outside the cache in every arrangement of the heads.

Tolerances as for the step's other tests: fp32 1e-5 (sums of 128 terms in
fp32), 16-bit outputs half a step of their type more."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNCore, GDNStateCache
from tests.gpu_util import DEV, assert_close, host, torch_dtype
from tests.test_gpu_serving import FP32, Case, ints, tol

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def most(fn):
    """fn(cu, slots) for 65535 sequences, all but four of them empty, and for
    the four alone: 65535 x 256 workgroups of 320 threads are more than 2^32
    threads.  Without a group the arrangement is the same, and so is every
    bit of the outputs and states."""
    N, at, lens = 65535, [0, 1, 40000, 65534], [3, 9, 1, 2]
    every, slots = np.zeros(N, np.int32), np.full(N, -1)
    every[at], slots[at] = lens, [4, 0, 2, 3]
    cu = lambda v: ints(np.concatenate([[0], np.cumsum(v)]))  # noqa: E731
    return fn(cu(lens), ints([4, 0, 2, 3])), fn(cu(every), ints(slots))


def test_the_rule_of_most_sequences_and_heads():
    hk, hv, d, T = 2, 256, 128, 15
    torch.manual_seed(1)
    core = GDNCore(CoreConfig(hk, hv, d), DEV)
    cache = GDNStateCache(core.cfg, 5, device=DEV)
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    q, k, v = (0.1 * r(T, hk * d)).to(BF), (0.1 * r(T, hk * d)).to(BF), r(T, hv * d).to(BF)
    g, beta = -torch.rand(T, hv, device=DEV), torch.rand(T, hv, device=DEV)
    cache.buffer.zero_()
    cache.S().normal_()
    start = cache.buffer.clone()

    def run(cu, slots):
        cache.buffer.copy_(start)
        o = core.recurrent(q, k, v, g, beta, cu, cache, slots)
        return o, cache.buffer.clone()

    few, many = most(run)
    assert bool(torch.isfinite(few[0]).all()) and not torch.equal(few[1], start)
    assert torch.equal(few[0], many[0]) and torch.equal(few[1], many[1])


def test_the_step_of_most_sequences_and_heads():
    h, d, T = 256, 128, 15
    torch.manual_seed(2)
    core = GDNCore(CoreConfig(h, h, d), DEV)
    C = core.cfg.channels
    cache = GDNStateCache(core.cfg, 5, device=DEV)
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    args = (r(T, C).to(BF), 0.25 * r(C, 4), r(T, h).to(BF), r(T, h).to(BF), -r(h).abs(), r(h), r(T, h, d).to(BF), 0.1 * r(d))
    cache.buffer.zero_()
    cache.S().normal_()
    cache.conv().normal_()
    start = cache.buffer.clone()

    def run(cu, slots):
        cache.buffer.copy_(start)
        out = core.step(*args, cu, cache, slots)
        return out, cache.buffer.clone()

    few, many = most(run)
    assert bool(torch.isfinite(few[0]).all()) and not torch.equal(few[1], start)
    assert torch.equal(few[0], many[0]) and torch.equal(few[1], many[1])


def step_in_64_bits(args, act, S_pool, C_pool, slot_in, slot_out, slot_tok, hk, hv, d):
    """The step from its definition, a sequence and a token at a time, in
    float64 on the device."""
    x, w, a, b, A, dt, z, wn, cu = args
    f, cu = torch.float64, cu.tolist()
    x, w, a, b, A, dt, z, wn = (t.to(f) for t in (x, w, a, b, A, dt, z, wn))
    S_new, C_new = S_pool.to(f), C_pool.to(f)
    head = torch.arange(hv, device=x.device) // (hv // hk)
    out = torch.zeros(x.shape[0], hv, d, dtype=f, device=x.device)
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    for n, (t0, t1) in enumerate(zip(cu, cu[1:])):
        fresh = slot_in[n] < 0
        S = torch.zeros(hv, d, d, dtype=f, device=x.device) if fresh else S_pool[slot_in[n]].to(f)
        rows = torch.zeros(3, x.shape[1], dtype=f, device=x.device) if fresh else C_pool[slot_in[n]].to(f)
        for t in range(t0, t1):
            win = torch.cat([rows, x[t:t + 1]])
            rows = win[1:]
            u = (win * w.t()).sum(0)
            y = u * torch.sigmoid(u)
            q, k = unit(y[:hk * d].view(hk, d))[head] * d ** -0.5, unit(y[hk * d:2 * hk * d].view(hk, d))[head]
            v = y[2 * hk * d:].view(hv, d)
            S = S * torch.exp(-torch.exp(A) * torch.logaddexp(a[t] + dt, torch.zeros_like(dt)))[:, None, None]
            delta = torch.sigmoid(b[t])[:, None] * (v - (S * k[:, None, :]).sum(2))
            S = S + delta[:, :, None] * k[:, None, :]
            o = (S * q[:, None, :]).sum(2)
            o = o / (o.square().mean(1, keepdim=True) + 1e-6).sqrt() * (1 + wn)
            out[t] = o * torch.sigmoid(z[t]) * (z[t] if act == 0 else 1)
            if slot_tok is not None and slot_tok[t] >= 0:
                S_new[slot_tok[t]], C_new[slot_tok[t]] = S, rows
        if slot_out[n] >= 0:
            S_new[slot_out[n]], C_new[slot_out[n]] = S, rows
    return out, S_new, C_new


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("dtype,hk,hv,lens", [
    ("bf16", 64, 128, [1, 9, 0, 17] + [1] * 29), ("bf16", 64, 192, [2, 20, 0, 1] + [1] * 29),
    ("fp16", 32, 160, [9, 1, 0, 3] + [1] * 61), ("fp32", 64, 192, [1, 8, 0, 10] + [1] * 29)])
def test_thousands_of_groups_of_large_heads(dtype, hk, hv, lens, drafts):
    """From 2048 groups on a workgroup takes its group's heads one by one:
    states pass from round to round, and q's and k's conv rows are written in
    the last."""
    d, N, T = 128, len(lens), sum(lens)
    assert N * hk >= 2048
    tdt = torch_dtype(dtype)
    torch.manual_seed(hv)
    core = GDNCore(CoreConfig(hk, hv, d, tdt), DEV)
    C = core.cfg.channels
    n_slots = N + (T if drafts else 0) + 2
    cache = GDNStateCache(core.cfg, n_slots, device=DEV)
    cache.buffer.zero_()
    cache.S().normal_(0, 0.3)
    cache.conv().normal_()
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    args = (r(T, C).to(tdt), 0.25 * r(C, 4), r(T, hv).to(tdt), r(T, hv).to(tdt), -1 - r(hv).abs(), 0.1 * r(hv),
            r(T, hv, d).to(tdt), 0.1 * r(d), ints(np.concatenate([[0], np.cumsum(lens)])))
    order = np.random.default_rng(hv).permutation(n_slots).tolist()
    slot_in = order[:N]
    slot_in[3] = -1                              # a new sequence
    slot_out, slot_tok = slot_in[:], None
    slot_out[3] = order[N]
    if drafts:
        slot_tok = [s if i % 4 else -1 for i, s in enumerate(order[N + 1:N + 1 + T])]
    want, S, conv = step_in_64_bits(args, 0, cache.S(), cache.conv(), slot_in, slot_out, slot_tok, hk, hv, d)
    got = core.step(*args, cache, ints(slot_in), ints(slot_out), ints(slot_tok) if drafts else None)
    assert_close("out", host(got), host(want), tol(dtype))
    # one comparison on the device: the states are gigabytes
    err = (cache.S().double() - S).abs().max() / S.abs().max()
    assert bool(torch.isfinite(cache.S()).all()) and float(err) <= FP32
    assert torch.equal(cache.conv().double(), conv)


@pytest.mark.parametrize("dtype,hk,hv,d,more", [
    ("bf16", 1, 4, 128, 0),        # heads apart over eight waves, the rows of q and k in a second launch
    ("bf16", 2, 16, 128, 20),      # heads apart over four waves
    ("fp32", 1, 5, 32, 0),         # apart, d = 32
    ("bf16", 4, 16, 128, 30),      # in rounds of two
    ("fp16", 2, 10, 128, 62),      # in rounds of three
    ("bf16", 3, 9, 32, 0)])        # three together
def test_bad_slots_in_every_arrangement(dtype, hk, hv, d, more):
    lens = [2, 1, 3, 9] + [1] * more
    N = len(lens)
    c = Case(dtype, hk, hv, d, lens, N + 1, seed=3)
    n = N + 1
    got = c.step([0, n, 1, 2] + list(range(4, N)), [0, 3, 1 << 30, 2] + list(range(4, N)))
    ref = c.ref([0, -1, -1, 2] + list(range(4, N)), [0, -1, -1, 2] + list(range(4, N)))
    assert bool(torch.isnan(got[2:6]).all())
    keep = [0, 1] + list(range(6, sum(lens)))
    assert_close("out", host(got)[keep], ref[0][keep], tol(dtype))
    assert_close("S", host(c.cache.S()), ref[1], FP32)
    assert np.array_equal(host(c.cache.conv()), ref[2])


@pytest.mark.parametrize("dtype,hk,hv,d", [("bf16", 1, 2, 128), ("bf16", 2, 66, 128), ("fp32", 1, 3, 32)])
def test_bad_slots_of_the_rule(dtype, hk, hv, d):
    """A head over four workgroups, one to a workgroup, and of 32 columns."""
    lens = [2, 1, 3, 9]
    T, tdt = sum(lens), torch_dtype(dtype)
    torch.manual_seed(4)
    core = GDNCore(CoreConfig(hk, hv, d, tdt), DEV)
    cache = GDNStateCache(core.cfg, 4, device=DEV)
    cache.buffer.zero_()
    cache.S().normal_()
    start = cache.buffer.clone()
    r = lambda *s: (0.2 * torch.randn(*s, device=DEV)).to(tdt)  # noqa: E731
    args = (r(T, hk * d), r(T, hk * d), r(T, hv * d), -torch.rand(T, hv, device=DEV), torch.rand(T, hv, device=DEV),
            ints(np.concatenate([[0], np.cumsum(lens)])), cache)
    want = core.recurrent(*args, ints([0, -1, -1, 2]), ints([0, -1, -1, 2]))
    after = cache.buffer.clone()
    cache.buffer.copy_(start)
    got = core.recurrent(*args, ints([0, 4, 1, 2]), ints([0, 3, 1 << 30, 2]))
    keep = [0, 1] + list(range(6, T))
    assert bool(torch.isnan(got[2:6]).all()) and bool(torch.isfinite(got[keep]).all())
    assert torch.equal(got[keep], want[keep]) and torch.equal(cache.buffer, after)
    assert not torch.equal(after, start)
