"""The recurrent form over cached states on the GPU: gdn_step_fwd,
gdn_recurrent_fwd and the slot tables, against the fp64 oracle run token by
token, and runs of the serving calls together.

Tolerances (max|got - ref| / max|ref| of a tensor).  Everything is computed in
fp32 from identical inputs and rounded once: sums of 128 terms are off by at
most 128 * 2^-24 = 7.6e-6 of their terms' sum and in practice by its square
root, so fp32 outputs and states are held to 1e-5; a 16-bit output adds half a
step of its type relative to the value, eps / 2 (bf16 2^-8, fp16 2^-11).
Conv rows are copies and compared exactly."""
import numpy as np
import pytest
import torch

import oracle
from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNCore, GDNLayer, GDNStateCache
from tests.gpu_util import DEV, assert_close, dev, host, torch_dtype

pytestmark = pytest.mark.gpu

FP32 = 1e-5


def tol(dtype):
    return FP32 if dtype == "fp32" else torch.finfo(torch_dtype(dtype)).eps / 2 + FP32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rnd(a, dtype):
    """Rounded to the storage type, as float64."""
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch_dtype(dtype)).double().numpy()


class Case:
    """Inputs of a step over a cache, on the host (float64, exact in the
    storage type) and on the device."""

    def __init__(self, dtype, hk, hv, d, lens, n_slots, seed=0, act=0, T=None, strided=False,
                 layers=1, layer=0):
        rng = np.random.default_rng(seed)
        self.dtype, self.hk, self.hv, self.d, self.act = dtype, hk, hv, d, act
        self.lens = lens
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T = int(self.cu[-1]) if T is None else T     # rows behind the last sequence: padding
        self.T = T
        C = self.C = 2 * hk * d + hv * d
        self.x = rnd(rng.standard_normal((T, C)), dtype)
        self.a = rnd(rng.standard_normal((T, hv)), dtype)
        self.b = rnd(rng.standard_normal((T, hv)), dtype)
        self.z = rnd(rng.standard_normal((T, hv, d)), dtype)
        f = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
        self.w_conv = f(0.25 * rng.standard_normal((C, 4)))
        self.A_log = f(np.log(rng.uniform(0.02, 0.3, hv)))
        self.dt_bias = f(0.1 * rng.standard_normal(hv))
        self.w_norm = f(0.1 * rng.standard_normal(d))
        self.S = f(0.3 * rng.standard_normal((n_slots, hv, d, d)))
        self.conv = rnd(rng.standard_normal((n_slots, 3, C)), dtype)
        tdt = torch_dtype(dtype)
        self.core = GDNCore(CoreConfig(hk, hv, d, tdt, act=act), DEV)
        self.cache = GDNStateCache(self.core.cfg, n_slots, n_layers=layers, device=DEV)
        self.layer = layer
        self.cache.buffer.fill_(0xFF)                # NaN wherever nothing is put
        self.cache.S(layer).copy_(dev(self.S))
        self.cache.conv(layer).copy_(dev(self.conv, tdt))
        if strided:                                  # columns of one wide projection
            W = C + hv * d + 2 * hv
            P = torch.full((T, (W + 7) // 8 * 8 + 8), float("nan"), dtype=tdt, device=DEV)
            self.t_x, self.t_z = P[:, :C], P[:, C:C + hv * d]
            self.t_a, self.t_b = P[:, C + hv * d:W - hv], P[:, W - hv:W]
            for t, h in ((self.t_x, self.x), (self.t_z, self.z.reshape(T, -1)), (self.t_a, self.a),
                         (self.t_b, self.b)):
                t.copy_(dev(h, tdt))
        else:
            self.t_x, self.t_z = dev(self.x, tdt), dev(self.z, tdt)
            self.t_a, self.t_b = dev(self.a, tdt), dev(self.b, tdt)
        self.t_w = [dev(v) for v in (self.w_conv, self.A_log, self.dt_bias, self.w_norm)]

    def args(self):
        w, A, dt, wn = self.t_w
        return self.t_x, w, self.t_a, self.t_b, A, dt, self.t_z, wn, ints(self.cu)

    def step(self, slot_in, slot_out=None, slot_tok=None):
        t = lambda v: None if v is None else ints(v)  # noqa: E731
        return self.core.step(*self.args(), self.cache, t(slot_in), t(slot_out), t(slot_tok),
                              layer=self.layer)

    def ref(self, slot_in, slot_out=None, slot_tok=None):
        """out [T, hv, d] and the cache after the call, from the oracle."""
        slot_out = slot_in if slot_out is None else slot_out
        hk, hv, d = self.hk, self.hv, self.d
        out = np.zeros((self.T, hv, d))
        S_new, C_new = self.S.copy(), self.conv.copy()
        for n in range(len(self.lens)):
            t0, t1 = self.cu[n], self.cu[n + 1]
            S = self.S[slot_in[n]] if slot_in[n] >= 0 else np.zeros((hv, d, d))
            rows = self.conv[slot_in[n]] if slot_in[n] >= 0 else np.zeros((3, self.C))
            for t in range(t0, t1):
                one = slice(t, t + 1)
                y, rows = oracle.conv_state_fwd(self.x[one], self.w_conv, [0, 1], 2 * hk * d, d,
                                                rows[None])
                rows = rows[0]
                g, beta = oracle.gate_fwd(self.a[one], self.b[one], self.A_log, self.dt_bias)
                q, k, v = (y[:, :hk * d].reshape(1, hk, d), y[:, hk * d:2 * hk * d].reshape(1, hk, d),
                           y[:, 2 * hk * d:].reshape(1, hv, d))
                o, S = oracle.delta_fwd(q, k, v, g, beta, [0, 1], d ** -0.5, S[None])
                S = S[0]
                out[t] = oracle.norm_fwd(o, self.z[one], self.w_norm, self.act)[0]
                if slot_tok is not None and slot_tok[t] >= 0:
                    S_new[slot_tok[t]], C_new[slot_tok[t]] = S, rows
            if slot_out[n] >= 0:
                S_new[slot_out[n]], C_new[slot_out[n]] = S, rows
        return out, S_new, C_new

    def check(self, got, ref, what=""):
        out, S, conv = ref
        T = int(self.cu[-1])
        if T:
            assert_close(what + "out", host(got)[:T], out[:T], tol(self.dtype))
        assert_close(what + "S", host(self.cache.S(self.layer)), S, FP32)
        assert np.array_equal(host(self.cache.conv(self.layer)), conv), what + "conv rows"
        untouched = [i for i in range(len(S)) if np.array_equal(S[i], self.S[i])]
        assert torch.equal(self.cache.S(self.layer)[untouched], dev(self.S[untouched])), what


CASES = {
    "decode_bf16": dict(dtype="bf16", hk=2, hv=6, d=128, lens=[1] * 5),
    "decode_one_bf16_full_heads": dict(dtype="bf16", hk=16, hv=48, d=128, lens=[1]),
    "ragged_bf16_strided": dict(dtype="bf16", hk=1, hv=4, d=128, lens=[1, 0, 3, 9, 17, 2], strided=True),
    "ragged_fp16": dict(dtype="fp16", hk=2, hv=2, d=128, lens=[8, 16, 7, 1]),
    "ragged_fp32": dict(dtype="fp32", hk=1, hv=2, d=128, lens=[1, 5, 33, 0], strided=True),
    "small_fp32": dict(dtype="fp32", hk=1, hv=2, d=32, lens=[1, 2, 3, 4, 0, 9]),
    "small_bf16_strided": dict(dtype="bf16", hk=3, hv=9, d=32, lens=[1] * 7, strided=True),
    "small_fp16_sigmoid": dict(dtype="fp16", hk=1, hv=8, d=32, lens=[2, 65, 1], act=1),
    "one_head_bf16_sigmoid": dict(dtype="bf16", hk=1, hv=1, d=128, lens=[4], act=1),
    # heads of a group in several rounds, the last not full; long enough to go apart, or not
    "five_of_a_group_bf16": dict(dtype="bf16", hk=1, hv=5, d=128, lens=[9, 1, 20, 3]),
    "four_of_a_group_fp32": dict(dtype="fp32", hk=2, hv=8, d=128, lens=[5, 11, 2, 7, 8, 1]),
    "seven_of_a_group_fp16_strided": dict(dtype="fp16", hk=1, hv=7, d=32, lens=[17, 0, 1], strided=True),
    "three_of_a_group_fp32_short": dict(dtype="fp32", hk=3, hv=9, d=128, lens=[1, 6, 0, 2]),
    # apart, with a head over eight waves, and (over 256 heads) over four
    "apart_fp32": dict(dtype="fp32", hk=1, hv=3, d=128, lens=[9, 17, 8]),
    "apart_fp16_strided": dict(dtype="fp16", hk=2, hv=8, d=128, lens=[12, 0, 15, 25], strided=True),
    "apart_many_heads_bf16": dict(dtype="bf16", hk=2, hv=16, d=128, lens=[8] * 19 + [12]),
    # too many groups for that: in rounds of two and of three
    "rounds_of_two_bf16": dict(dtype="bf16", hk=4, hv=16, d=128, lens=[1, 2, 0, 9] + [1] * 30),
    "rounds_of_two_fp32": dict(dtype="fp32", hk=4, hv=16, d=32, lens=[3, 10, 0, 1] + [1] * 30, strided=True),
    "rounds_of_three_fp16": dict(dtype="fp16", hk=2, hv=10, d=128, lens=[17, 0, 2] + [1] * 63),
    "rounds_of_three_fp32": dict(dtype="fp32", hk=2, hv=10, d=128, lens=[9, 0, 2] + [1] * 63, act=1),
    "rounds_of_three_bf16": dict(dtype="bf16", hk=4, hv=20, d=32, lens=[2, 0, 17] + [1] * 31, strided=True),
    # a few thousand groups
    "many_bf16": dict(dtype="bf16", hk=2, hv=4, d=32, lens=[1] * 1000 + [2] * 40),
    "three_together_fp16": dict(dtype="fp16", hk=2, hv=6, d=32, lens=[1, 9, 0, 2, 7]),
    "five_of_a_group_fp32_strided": dict(dtype="fp32", hk=2, hv=10, d=32, lens=[3, 8, 1, 0], strided=True),
    "many_of_three_bf16": dict(dtype="bf16", hk=4, hv=12, d=32, lens=[1] * 520 + [0] * 5 + [3] * 4),
    "most_heads_bf16": dict(dtype="bf16", hk=1, hv=256, d=32, lens=[1, 2]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("mode", ["inplace", "elsewhere", "drafts", "nowhere"])
def test_step_matches_the_oracle(name, mode):
    kw = CASES[name]
    N, T = len(kw["lens"]), sum(kw["lens"])
    n_slots = 2 * N + T + 2
    c = Case(n_slots=n_slots, seed=len(name), **kw)
    order = np.random.default_rng(5).permutation(n_slots).tolist()
    slot_in, slot_out, slot_tok = order[:N], order[N:2 * N], order[2 * N:2 * N + T]
    if N > 1:
        slot_in[1] = -1                          # a new sequence
    if mode == "inplace":
        slot_out, slot_tok = None, None
    elif mode == "elsewhere":
        slot_tok = None
        if N > 2:
            slot_in[2] = slot_in[0]              # two sequences continue from one slot
    elif mode == "nowhere":
        slot_out, slot_tok = [-1] * N, None
    else:
        slot_tok = [s if i % 3 else -1 for i, s in enumerate(slot_tok)]
    got = c.step(slot_in, slot_out, slot_tok)
    c.check(got, c.ref(slot_in, slot_out, slot_tok))


CASES_RULE = dict(CASES, many_heads_bf16=dict(dtype="bf16", hk=1, hv=64, d=128, lens=[1, 3, 9, 0, 1]),
                  many_heads_fp32=dict(dtype="fp32", hk=64, hv=64, d=128, lens=[2, 1, 1, 1, 10]))


@pytest.mark.parametrize("name", ["decode_bf16", "ragged_fp16", "ragged_fp32", "small_fp32", "small_bf16_strided",
                                  "many_heads_bf16", "many_heads_fp32"])
@pytest.mark.parametrize("drafts", [False, True])
def test_recurrent_matches_the_oracle(name, drafts):
    """The rule alone, q, k, v as columns of one tensor."""
    kw = CASES_RULE[name]
    dtype, hk, hv, d, lens = (kw[x] for x in ("dtype", "hk", "hv", "d", "lens"))
    N, T = len(lens), sum(lens)
    rng = np.random.default_rng(7)
    y = rng.standard_normal((T, 2 * hk + hv, d))
    y[:, :2 * hk] /= np.linalg.norm(y[:, :2 * hk], axis=-1, keepdims=True)
    y = rnd(y, dtype)
    g = np.float32(-rng.uniform(0, 0.3, (T, hv))).astype(np.float64)
    beta = np.float32(rng.uniform(0, 1, (T, hv))).astype(np.float64)
    n_slots = N + T + 1
    S = np.float32(0.3 * rng.standard_normal((n_slots, hv, d, d))).astype(np.float64)
    slots = rng.permutation(n_slots).tolist()
    slot_in, slot_tok = slots[:N], (slots[N:N + T] if drafts else None)
    slot_in[0] = -1
    slot_out = slot_in[:]
    slot_out[0] = slots[N + T]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    S_ref, o_ref = S.copy(), np.zeros((T, hv, d))
    for n in range(N):
        st = S[slot_in[n]] if slot_in[n] >= 0 else np.zeros((hv, d, d))
        for t in range(cu[n], cu[n + 1]):
            q, k, v = y[t:t + 1, :hk], y[t:t + 1, hk:2 * hk], y[t:t + 1, 2 * hk:]
            o, st = oracle.delta_fwd(q, k, v, g[t:t + 1], beta[t:t + 1], [0, 1], d ** -0.5, st[None])
            o_ref[t], st = o[0], st[0]
            if drafts:
                S_ref[slot_tok[t]] = st
        S_ref[slot_out[n]] = st
    tdt = torch_dtype(dtype)
    core = GDNCore(CoreConfig(hk, hv, d, tdt), DEV)
    cache = GDNStateCache(core.cfg, n_slots, device=DEV)
    cache.S().copy_(dev(S))
    ty = dev(y.reshape(T, -1), tdt)
    o = core.recurrent(*core.split(ty), dev(g), dev(beta), ints(cu), cache, ints(slot_in), ints(slot_out),
                       ints(slot_tok) if drafts else None)
    assert_close("o", host(o), o_ref, tol(dtype))
    assert_close("S", host(cache.S()), S_ref, FP32)


@pytest.mark.parametrize("dtype,hk,hv,d", [("bf16", 2, 6, 128), ("fp32", 1, 3, 32), ("fp16", 1, 4, 128)])
def test_tokens_one_by_one_equal_one_call(dtype, hk, hv, d):
    """A token's arithmetic does not depend on how the tokens are cut into
    calls: outputs, states and conv rows agree bit by bit."""
    lens = [19, 5]
    c = Case(dtype, hk, hv, d, lens, 4, seed=3)
    args = c.args()
    start = c.cache.buffer.clone()
    slots = ints([2, 1])
    whole = c.core.step(*args, c.cache, slots)
    after = c.cache.buffer.clone()
    c.cache.buffer.copy_(start)
    for j in range(max(lens)):
        rows = [int(c.cu[n]) + j for n in range(2) if j < lens[n]]
        pick = lambda t: t[rows].contiguous()  # noqa: E731
        x, w, a, b, A, dt, z, wn, _ = args
        out = c.core.step(pick(x), w, pick(a), pick(b), A, dt, pick(z), wn,
                          ints(list(range(len(rows) + 1))), c.cache, slots[:len(rows)].contiguous())
        assert torch.equal(out, whole[rows]), j
    assert torch.equal(c.cache.S(), after[:, :c.cache.S()[0].numel() * 4].view(torch.float32)
                       .view_as(c.cache.S()))
    assert torch.equal(c.cache.buffer, after)


@pytest.mark.parametrize("hk,hv,d,N", [(4, 16, 128, 40), (2, 6, 128, 100), (1, 5, 32, 300), (16, 32, 128, 160)])
def test_runs_repeat_bit_by_bit(hk, hv, d, N):
    """The same call on the same states, again and again: helper and state
    waves meet at their barriers whichever is ahead."""
    torch.manual_seed(N)
    core = GDNCore(CoreConfig(hk, hv, d), DEV)
    cache = GDNStateCache(core.cfg, N, device=DEV)
    lens = [1 + (7 * n) % 20 for n in range(N)]
    T, C, bf = sum(lens), core.cfg.channels, torch.bfloat16
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    args = (r(T, C).to(bf), 0.25 * r(C, 4), r(T, hv).to(bf), r(T, hv).to(bf), -r(hv).abs(), r(hv), r(T, hv, d).to(bf),
            0.1 * r(d), ints(np.concatenate([[0], np.cumsum(lens)])))
    cache.buffer.zero_()
    cache.S().normal_()
    cache.conv().normal_()
    start, slots = cache.buffer.clone(), ints(np.random.default_rng(0).permutation(N))
    want = core.step(*args, cache, slots)
    after = cache.buffer.clone()
    assert bool(torch.isfinite(want).all())
    for k in range(25):
        cache.buffer.copy_(start)
        got = core.step(*args, cache, slots)
        assert torch.equal(got, want) and torch.equal(cache.buffer, after), k


def test_no_tokens_pass_states_through():
    c = Case("bf16", 1, 2, 128, [0, 0, 0], 5)
    got = c.step([0, 3, -1], [1, 3, 4])
    assert got.shape[0] == 0
    S, conv = c.S.copy(), c.conv.copy()
    S[1], conv[1], S[4], conv[4] = S[0], conv[0], 0, 0
    assert np.array_equal(host(c.cache.S()), S) and np.array_equal(host(c.cache.conv()), conv)
    rule = Case("bf16", 1, 2, 128, [0, 0], 3)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    f = torch.empty(0, 2, device=DEV)
    rule.core.recurrent(e[:, :128], e[:, :128], e, f, f, ints([0, 0, 0]), rule.cache, ints([2, -1]), ints([0, -1]))
    S = rule.S.copy()
    S[0] = S[2]
    assert np.array_equal(host(rule.cache.S()), S)


def test_padded_batch_leaves_the_rest_alone():
    """Rows behind the last sequence and the slots of padding stay as they
    were, whatever they hold."""
    c = Case("bf16", 2, 4, 128, [2, 1, 0, 0], 4, T=7)
    for t in (c.t_x, c.t_a, c.t_b, c.t_z):
        t[3:] = float("nan")
    sh = c.core.shape(7, 4)
    out = torch.full((7, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    x, w, a, b, A, dt, z, wn, cu = c.args()
    slots = [1, 2, -1, -1]
    L.gdn_step_fwd(sh, x, w, a, b, A, dt, z.view(7, -1), wn, 128 ** -0.5, c.cache.layer(), ints(slots),
                   ints(slots), None, cu, out)
    assert bool((out[3:] == 7).all())
    c.check(out, c.ref(slots))


def test_slots_outside_the_cache():
    """NaN rows and no state written for the sequences that name one; the
    others are computed as ever."""
    c = Case("fp16", 1, 2, 128, [2, 1, 3, 1], 4)
    got = c.step([0, 4, 1, 2], [0, 3, 1 << 30, 2])
    ref = c.ref([0, -1, -1, 2], [0, -1, -1, 2])
    assert bool(torch.isnan(got[2:6]).all()) and not bool(torch.isnan(got[:2]).any())
    keep = [0, 1, 6]
    assert_close("out", host(got)[keep], ref[0][keep], tol("fp16"))
    assert_close("S", host(c.cache.S()), ref[1], FP32)
    assert np.array_equal(host(c.cache.conv()), ref[2])
    d = Case("fp16", 1, 2, 128, [2, 1], 4)       # a bad slot_tok entry writes nothing
    got = d.step([0, 1], None, [7, 2, 4])
    d.check(got, d.ref([0, 1], None, [-1, 2, -1]))


def test_other_slots_do_not_leak():
    """A new sequence next to NaN and infinite states: zero means zero."""
    c = Case("bf16", 1, 2, 128, [3, 1], 3)
    ref = c.ref([-1, 2], [1, 2])
    c.cache.S()[0] = float("nan")
    c.cache.S()[1] = float("inf")
    c.cache.conv()[:2] = float("nan")
    got = c.step([-1, 2], [1, 2])
    assert_close("out", host(got), ref[0], tol("bf16"))
    assert_close("S", host(c.cache.S())[1:], ref[1][1:], FP32)
    assert np.array_equal(host(c.cache.conv())[1:], ref[2][1:])
    assert bool(torch.isnan(c.cache.S()[0]).all())


def test_extreme_gates():
    """Full decay (g = -inf from a = +inf keeps only the new write), no decay
    and beta 0 or 1."""
    c = Case("fp32", 1, 2, 32, [4], 1)
    c.a[:, 0], c.a[:, 1] = [1e30, -1e30, 80, -80], [-200, 3e4, 0, -1e30]
    c.b[:, 0], c.b[:, 1] = [200, -200, 1e30, -1e30], [0, 90, -90, 5]
    c.a, c.b = rnd(c.a, "fp32"), rnd(c.b, "fp32")
    c.t_a, c.t_b = dev(c.a), dev(c.b)
    got = c.step([0])
    c.check(got, c.ref([0]))


def test_large_unnormalised_values_in_fp32():
    """The recurrence has no 16-bit operands: values far beyond fp16's range."""
    hk, hv, d, T = 1, 2, 128, 3
    rng = np.random.default_rng(1)
    y = rng.standard_normal((T, 4, d))
    y[:, :2] /= np.linalg.norm(y[:, :2], axis=-1, keepdims=True)
    y[:, 2:] *= 1e9
    y = rnd(y, "bf16")
    g, beta = np.full((T, hv), -0.125), np.full((T, hv), 0.5)
    S = np.float32(1e9 * rng.standard_normal((1, hv, d, d))).astype(np.float64)
    o_ref, S_ref = oracle.delta_fwd(y[:, :1], y[:, 1:2], y[:, 2:], g, beta, [0, T], d ** -0.5, S)
    core = GDNCore(CoreConfig(hk, hv, d), DEV)
    cache = GDNStateCache(core.cfg, 1, device=DEV)
    cache.S().copy_(dev(S))
    o = core.recurrent(*core.split(dev(y.reshape(T, -1), torch.bfloat16)), dev(g), dev(beta), ints([0, T]),
                       cache, ints([0]))
    assert_close("o", host(o), o_ref, tol("bf16"))
    assert_close("S", host(cache.S()), S_ref, FP32)


def test_slots_far_apart():
    """Slot offsets beyond 2^32 bytes and 2^31 elements."""
    c = Case("bf16", 1, 2, 128, [1, 2], 4)
    gap = 3 << 30                                  # bytes between slots
    big = torch.empty(3 * gap + (1 << 20), dtype=torch.uint8, device=DEV)
    S = torch.as_strided(big.view(torch.float32), (4, 2, 128, 128), (gap // 4, 16384, 128, 1))
    at = 2 * 16384 * 4
    conv = torch.as_strided(big[at:].view(torch.bfloat16), (4, 3, c.C), (gap // 2, c.C, 1))
    L.gdn_cache_copy(c.cache.S(), S)
    L.gdn_cache_copy(c.cache.conv(), conv)
    x, w, a, b, A, dt, z, wn, cu = c.args()
    out = torch.empty((3, 2, 128), dtype=torch.bfloat16, device=DEV)
    L.gdn_step_fwd(c.core.shape(3, 2), x, w, a, b, A, dt, z.view(3, -1), wn, 128 ** -0.5,
                   L.make_cache(S, conv), ints([3, 1]), ints([3, 2]), None, cu, out)
    L.gdn_cache_copy(S, c.cache.S())
    L.gdn_cache_copy(conv, c.cache.conv())
    c.check(out, c.ref([3, 1], [3, 2]))


def test_another_layer_of_the_slots():
    c = Case("bf16", 1, 3, 128, [1, 4], 3, layers=3, layer=1)
    before = c.cache.buffer.clone()
    got = c.step([2, 0])
    c.check(got, c.ref([2, 0]))
    for k in (0, 2):
        n = c.cache.slot_bytes // 3
        assert torch.equal(c.cache.buffer[:, k * n:(k + 1) * n], before[:, k * n:(k + 1) * n])


@pytest.mark.parametrize("hk,hv,lens", [(1, 6, [3, 1, 2]), (1, 5, [20, 13]), (2, 4, [1, 9])])
def test_a_state_kept_in_the_slot_it_came_from(hk, hv, lens):
    """A single token's state may go to the slot that the sequence began from
    (its last goes elsewhere), heads together, in rounds and apart."""
    N, T = len(lens), sum(lens)
    c = Case("bf16", hk, hv, 128, lens, 2 * N, seed=8)
    slot_in, slot_out, tok = list(range(N)), list(range(N, 2 * N)), [-1] * T
    for n in range(N):
        tok[int(c.cu[n])] = n                       # after its first token
    got = c.step(slot_in, slot_out, tok)
    c.check(got, c.ref(slot_in, slot_out, tok))


@pytest.mark.parametrize("dtype,hk,hv,d,lens", [("bf16", 2, 6, 128, [1, 3, 9, 0]), ("fp32", 1, 4, 32, [5, 1, 1, 2]),
                                                ("fp16", 1, 5, 128, [17, 20, 1, 0])])
def test_nothing_is_written_outside(dtype, hk, hv, d, lens):
    """Bands of a known pattern around the cache, its workspace, the outputs
    and the tables stay as they were, through every serving call."""
    tdt, N, T = torch_dtype(dtype), len(lens), sum(lens)
    bands = []

    def banded(n, kind=torch.uint8):
        n *= torch.empty(0, dtype=kind).element_size()
        whole = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        bands.append(whole)
        return whole[4096:4096 + n].view(kind)

    c = Case(dtype, hk, hv, d, lens, 6)
    size, cfg = c.cache.slot_bytes, c.core.cfg
    refs = banded(6, torch.int32)
    refs.copy_(ints([1, 1, 2, 1, 0, 0]))
    cache = GDNStateCache(cfg, 6, device=DEV, buffer=banded(6 * size).view(6, size), refs=refs)
    cache.buffer.copy_(c.cache.buffer)
    x, w, a, b, A, dt, z, wn, cu = c.args()
    out = banded(T * hv * d, tdt)
    slots, tok, table, dst, remap = (banded(n, torch.int32) for n in (N, T, 9, 3, 6))
    slots.copy_(ints([0, 1, 2, 3]))
    tok.copy_(ints([4, 5] + [-1] * (T - 2)))
    sh = c.core.shape(T, N)
    L.gdn_step_fwd(sh, x, w, a, b, A, dt, z, wn, 1.0, cache.layer(), slots, slots, tok, cu, out)
    q, k, v = c.core.split(x)
    g, beta = -torch.rand(T, hv, device=DEV), torch.rand(T, hv, device=DEV)
    L.gdn_recurrent_fwd(sh, q, k, v, g, beta, 1.0, cache.layer(), slots, slots, tok, cu, out)
    ws = banded(L.gdn_cache_workspace(6))
    L.gdn_cache_fork(cache.buffer, refs, ints([2, -1, 0]), dst, ws)
    assert dst.tolist() == [4, 5, -1]
    cache.release(ints([0, 2, 5]))
    table.copy_(ints([0, 1, 2, 3, 4, 5, -1, 6, 3]))
    L.gdn_cache_compact(cache.buffer, refs, remap, table, ws)
    assert remap.tolist() == [-1, 1, 2, 3, 0, -1] and table.tolist() == [-1, 1, 2, 3, 0, -1, -1, 6, 3]
    cache.copy(ints([3, -1]), ints([4, 5]))
    torch.cuda.synchronize()
    for i, whole in enumerate(bands):
        assert bool((whole[:4096] == 0xA5).all()) and bool((whole[-4096:] == 0xA5).all()), i


def test_no_tables_at_all():
    """Without tables every sequence is new and no state is kept."""
    c = Case("bf16", 2, 4, 128, [2, 1, 5], 2)
    before = c.cache.buffer.clone()
    got = c.core.step(*c.args(), c.cache, None)
    c.check(got, c.ref([-1] * 3, [-1] * 3))
    q, k, v = (torch.randn(8, n, device=DEV).bfloat16() for n in (256, 256, 512))
    g, beta = -torch.rand(8, 4, device=DEV), torch.rand(8, 4, device=DEV)
    a = c.core.recurrent(q, k, v, g, beta, ints(c.cu), c.cache, None)
    b = c.core.recurrent(q, k, v, g, beta, ints(c.cu), c.cache, ints([-1] * 3), ints([-1] * 3), ints([-1] * 8))
    assert torch.equal(a, b) and torch.equal(c.cache.buffer, before)


def test_lengths_outside_the_tokens_are_clamped():
    c = Case("bf16", 1, 3, 128, [2, 2, 0, 0], 4)
    x, w, a, b, A, dt, z, wn, _ = c.args()
    slots = ints([3, 1, 0, 2])
    got = c.core.step(x, w, a, b, A, dt, z, wn, ints([-9, 2, 1 << 30, 1, -(1 << 31)]), c.cache, slots)
    c.check(got, c.ref([3, 1, 0, 2]))


def test_as_many_sequences_as_a_call_takes():
    """65535 sequences of one token, against the formula in elementary torch."""
    N, d = 65535, 32
    torch.manual_seed(3)
    core = GDNCore(CoreConfig(1, 1, d, torch.float32, scale=1.0), DEV)
    cache = GDNStateCache(core.cfg, N, device=DEV)
    cache.S().normal_()
    q, k, v = (torch.randn(N, d, device=DEV) for _ in range(3))
    k /= k.norm(dim=1, keepdim=True)
    g, beta = -torch.rand(N, 1, device=DEV), torch.rand(N, 1, device=DEV)
    S = cache.S()[:, 0].double() * torch.exp(g.double())[..., None]
    delta = beta.double() * (v.double() - (S * k.double()[:, None]).sum(2))
    S = S + delta[..., None] * k.double()[:, None]
    want = (S * q.double()[:, None]).sum(2)
    slots = torch.arange(N, dtype=torch.int32, device=DEV)
    o = core.recurrent(q, k, v, g, beta, torch.arange(N + 1, dtype=torch.int32, device=DEV), cache, slots)
    assert_close("o", host(o[:, 0]), host(want), FP32)
    assert_close("S", host(cache.S()[:, 0]), host(S), FP32)


def test_on_a_given_stream():
    c = Case("bf16", 2, 4, 128, [1, 3], 2)
    want = c.ref([1, 0])
    x, w, a, b, A, dt, z, wn, cu = c.args()
    out, slots = torch.empty(4, 4, 128, dtype=torch.bfloat16, device=DEV), ints([1, 0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    L.gdn_step_fwd(c.core.shape(4, 2), x, w, a, b, A, dt, z.view(4, -1), wn, 128 ** -0.5, c.cache.layer(), slots,
                   slots, None, cu, out, stream=st)
    st.synchronize()
    c.check(out, want)


def test_on_another_stream():
    c = Case("bf16", 2, 4, 128, [1] * 6, 6)
    want = c.ref([5, 4, 3, 2, 1, 0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = c.step([5, 4, 3, 2, 1, 0])
    st.synchronize()
    c.check(got, want)


def test_two_caches_on_two_streams():
    cs = [Case("bf16", 2, 4, 128, [1] * 40 + [3] * 5, 45, seed=s) for s in (1, 2)]
    slots = list(range(45))
    want = [c.ref(slots) for c in cs]
    args = [(c.args(), ints(slots)) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [None, None]
    for i in (0, 1):
        with torch.cuda.stream(streams[i]):
            got[i] = cs[i].core.step(*args[i][0], cs[i].cache, args[i][1])
    torch.cuda.synchronize()
    for c, g, w in zip(cs, got, want):
        c.check(g, w)


def test_captured_and_replayed_with_other_batches():
    """One graph of a step for a padded batch, replayed with other lengths,
    slots and inputs; every replay equals the eager call."""
    T, N = 12, 6
    c = Case("bf16", 2, 4, 128, [1] * N, 8, T=T)
    x, w, a, b, A, dt, z, wn, _ = c.args()
    cu, si, so, st = ints([0] * (N + 1)), ints([-1] * N), ints([-1] * N), ints([-1] * T)
    args = (x, w, a, b, A, dt, z, wn, cu, c.cache, si, so, st)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.core.step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.core.step(*args)
    rng = np.random.default_rng(4)
    for k in range(4):
        lens = [[1, 1, 1, 1, 1, 1], [3, 0, 2, 1, 0, 0], [1, 0, 0, 0, 0, 0], [4, 4, 4, 0, 0, 0]][k]
        slots = rng.permutation(8)[:N].tolist()
        cu.copy_(ints(np.concatenate([[0], np.cumsum(lens)])))
        si.copy_(ints([s if n else -1 for s, n in zip(slots, lens)]))
        so.copy_(si)
        used = [s for s, n in zip(slots, lens) if n]
        free = [s for s in range(8) if s not in used]
        tok = [-1] * T
        tok[0] = free[0]
        st.copy_(ints(tok))
        for t in (x, a, b, z):
            t.normal_()
        before = c.cache.buffer.clone()
        graph.replay()
        torch.cuda.synchronize()
        got, after = out.clone(), c.cache.buffer.clone()
        c.cache.buffer.copy_(before)
        eager = c.core.step(*args)
        n = sum(lens)
        assert torch.equal(got[:n], eager[:n]), k
        assert torch.equal(after, c.cache.buffer), k
        assert not torch.equal(after, before), k


def test_check_slots_finds_each_fault():
    core = GDNCore(CoreConfig(1, 2, 32, check_slots=True), DEV)
    cache = GDNStateCache(core.cfg, 20000, device=DEV)     # more than one range of the check

    def run(lens, si, so, tok=None):
        T = sum(lens)
        cu = ints(np.concatenate([[0], np.cumsum(lens)]))
        t = lambda v: None if v is None else ints(v)  # noqa: E731
        core.check_slots(core.shape(T, len(lens)), cache, t(si), t(so), t(tok), cu)

    run([1, 2], [0, 19999], [0, 19999])
    run([1, 2], [5, 5], [6, 19999], [-1, 9000, 5000])
    run([1, 0], None, None)
    run([2, 0], [-1, -1], [-1, -1], [-1, -1])
    for bad, args in (("outside", ([1, 1], [0, 20000], [0, 1])), ("outside", ([1, 1], [0, 1], [0, 1 << 30])),
                      ("outside", ([1, 1], [0, 1], [0, 1], [2, 20000])),
                      ("twice", ([1, 1], [0, 1], [9001, 9001])), ("twice", ([1, 1], [0, 1], [0, 1], [19999, 19999])),
                      ("twice", ([1, 1], [0, 1], [0, 1], [0, -1])),
                      ("read by another", ([1, 1], [0, 1], [1, 2])),
                      ("read by another", ([1, 1], [0, 19999], [0, 2], [19999, -1]))):
        with pytest.raises(ValueError, match=bad):
            run(*args)
    with pytest.raises(ValueError, match="twice"):
        z = torch.zeros(2, 128, dtype=torch.bfloat16, device=DEV)
        f = torch.zeros(2, 2, device=DEV)
        core.recurrent(z[:, :32], z[:, :32], z[:, :64], f, f, ints([0, 1, 2]), cache, ints([0, 1]), ints([3, 3]))


def test_prefill_then_steps_then_drafts():
    """A run of the serving calls: prompts go in by the chunked form, a
    sequence forks, tokens follow one at a time, drafts are checked and partly
    refused, a sequence ends, the cache is compacted, and the others go on.
    The outputs are those of the whole token rows in one pass of the oracle."""
    hk, hv, d, dtype = 2, 4, 128, "bf16"
    lens = [150, 70, 3]
    total = 24                                          # tokens after each prompt, at most
    rng = np.random.default_rng(11)
    big = Case(dtype, hk, hv, d, [n + total for n in lens], 1, seed=11)
    core, w = big.core, big.t_w
    cache = GDNStateCache(core.cfg, 8, device=DEV)
    cache.buffer.fill_(0xFF)
    base = big.cu[:-1].tolist()

    def rows(idx):
        i = torch.tensor(idx, device=DEV)
        return big.t_x[i], w[0], big.t_a[i], big.t_b[i], w[1], w[2], big.t_z[i], w[3]

    ref, _, _ = big.ref([-1] * 3, [-1] * 3)

    def same(got, idx):
        # chunked outputs follow the training path's bar, single tokens after it too: its
        # state carries the chunked form's 16-bit rounding
        assert_close("out", host(got), ref[idx], 5e-3)

    slots = cache.fork(ints([-1, -1, -1]))
    assert slots.tolist() == [0, 1, 2]
    idx = [base[n] + t for n in range(3) for t in range(lens[n])]
    same(core.prefill(*rows(idx), ints(np.concatenate([[0], np.cumsum(lens)])), cache, slots), idx)
    at = lens[:]
    for _ in range(5):                                  # one token each
        idx = [base[n] + at[n] for n in range(3)]
        same(core.step(*rows(idx), ints([0, 1, 2, 3]), cache, slots), idx)
        at = [t + 1 for t in at]
    twin = cache.fork(slots[:1].contiguous())           # sequence 0 goes on twice
    assert twin.tolist() == [3]
    drafts = cache.fork(ints([-1] * 4))                 # room for four drafts' states
    assert drafts.tolist() == [4, 5, 6, 7]
    idx = [base[0] + at[0] + j for j in range(4)]
    one = ints([0, 4])
    same(core.step(*rows(idx), one, cache, slots[:1].contiguous(), ints([-1]), drafts), idx)
    cache.copy(drafts[1:2].contiguous(), slots[:1].contiguous())    # two drafts are taken
    cache.release(drafts)
    at[0] += 2
    same(core.step(*rows([base[0] + at[0]]), ints([0, 1]), cache, slots[:1].contiguous()), [base[0] + at[0]])
    at[0] += 1
    cache.release(slots[1:2].contiguous())              # sequence 1 ends
    table = torch.cat([slots, twin])
    cache.compact(table)
    assert table.tolist() == [0, -1, 2, 1]
    assert cache.refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    live = table[[0, 2, 3]].contiguous()
    twin_at = lens[0] + 5
    for _ in range(3):
        idx = [base[0] + at[0], base[2] + at[2], base[0] + twin_at]
        same(core.step(*rows(idx), ints([0, 1, 2, 3]), cache, live), idx)
        at[0], at[2], twin_at = at[0] + 1, at[2] + 1, twin_at + 1


def test_prefill_passes_slots_as_step_does():
    """Empty and new sequences, and slots outside the cache."""
    c = Case("bf16", 1, 2, 128, [5, 0, 70, 4], 6, seed=2)
    slot_in, slot_out = [0, 1, -1, 6], [0, 2, 3, 4]
    x, w, a, b, A, dt, z, wn, cu = c.args()
    got = c.core.prefill(x, w, a, b, A, dt, z, wn, cu, c.cache, ints(slot_in), ints(slot_out))
    out, S, conv = c.ref(slot_in[:3] + [-1], slot_out)
    assert_close("out", host(got)[:75], out[:75], 5e-3)
    assert bool(torch.isnan(got[75:]).all()) and bool(torch.isnan(c.cache.S()[4]).all())
    keep = [0, 1, 2, 3, 5]
    assert_close("S", host(c.cache.S())[keep], S[keep], 5e-3)
    assert np.array_equal(host(c.cache.S())[2], c.S[1])
    assert np.array_equal(host(c.cache.conv())[keep], conv[keep])


def test_layer_step_follows_layer_forward():
    """The layer with its projections: tokens one by one after a prompt equal
    the whole forward (library products of other sizes and 16-bit roundings
    between them: the training path's bar)."""
    torch.manual_seed(0)
    H, hk, hv, d, T = 256, 1, 2, 128, 40
    cfg = CoreConfig(hk, hv, d)
    C = cfg.channels
    W = {n: (torch.randn(o, i, device=DEV) / i ** 0.5).bfloat16()
         for n, o, i in (("x", C, H), ("z", hv * d, H), ("a", hv, H), ("b", hv, H), ("out", H, hv * d))}
    layer = GDNLayer(cfg, H, W, DEV)
    X = torch.randn(T, H, device=DEV).bfloat16()
    w_conv = 0.25 * torch.randn(C, 4, device=DEV)
    A_log, dt, wn = torch.log(torch.tensor([0.1, 0.3], device=DEV)), torch.zeros(hv, device=DEV), torch.zeros(d, device=DEV)
    want = layer.forward(X, w_conv, A_log, dt, wn, ints([0, T]))["Y"]
    cache = GDNStateCache(cfg, 2, n_layers=2, device=DEV)
    slot = cache.fork(ints([-1]))
    got = [layer.step(X[:30], w_conv, A_log, dt, wn, ints([0, 30]), cache, slot, layer=1)]
    got += [layer.step(X[t:t + 1], w_conv, A_log, dt, wn, ints([0, 1]), cache, slot, layer=1) for t in range(30, T)]
    assert_close("Y", host(torch.cat(got)), host(want), 1e-2)
