"""The operators of a model's block together, as they are used: norm,
projections and core of a served layer over its cached states, and the norm
around the layer in training."""
import numpy as np
import pytest
import torch

import oracle
from gated_deltanet_layer_causal_amd import inputs as gi
from gated_deltanet_layer_causal_amd.block import GDNLayer4, Linear4, ResidualNorm
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNLayer, GDNStateCache
from tests.gpu_util import DEV, FWD_TOL_BF16, GRAD_TOL_BF16, assert_close, host

pytestmark = pytest.mark.gpu

HK, HV, D, H = 2, 4, 128, 320
CFG = dict(hk=HK, hv=HV, d=D, dtype=torch.bfloat16)


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    C = 2 * HK * D + HV * D
    dims = {"x": (C, H), "z": (HV * D, H), "a": (HV, H), "b": (HV, H), "out": (H, HV * D)}
    return {k: (torch.randn(s, generator=g) * s[1] ** -0.5).to(torch.bfloat16).to(DEV) for k, s in dims.items()}


def params(seed):
    g = torch.Generator().manual_seed(seed + 50)
    C = 2 * HK * D + HV * D
    return {"w_conv": torch.randn(C, 4, generator=g) * 0.5, "A_log": torch.rand(HV, generator=g) - 2,
            "dt_bias": torch.randn(HV, generator=g) * 0.1, "w_norm": torch.randn(D, generator=g) * 0.1}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def values4(layer4):
    """The layer's weights as their 4-bit values, name -> [out, in]."""
    W = layer4.proj_in.weight(torch.float32)
    W = {k: v.t() for k, v in zip(("x", "z", "a", "b"), layer4.split(W.t()))}
    W["out"] = layer4.proj_out.weight(torch.float32)
    return W


@pytest.mark.parametrize("eight", [False, True])
def test_served_layer_against_the_oracle(eight):
    """Prompts, then tokens one by one and in pieces: norm -> projections ->
    core -> projection against one pass of the oracle over the norm's rows as
    the products take them (rounded to bf16, or their values in 8 bits)."""
    W, p = weights(1), params(1)
    layer = GDNLayer4(CoreConfig(**CFG), H, W)
    norm = ResidualNorm(H, eps=1e-6)
    lens, N = [9, 5, 12], 3
    cu = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator().manual_seed(2)
    x, res = ((torch.randn(cu[-1], H, generator=g) * s).to(torch.bfloat16).to(DEV) for s in (1.0, 3.0))
    w = (torch.randn(H, generator=g) * 0.1).to(DEV)
    pd = {k: v.to(DEV) for k, v in p.items()}
    cache = GDNStateCache(layer.cfg, 4)
    slots = ints([2, 0, 3])
    cache.buffer.fill_(255)
    Y = torch.empty(int(cu[-1]), H, dtype=torch.bfloat16, device=DEV)
    rows = torch.empty(int(cu[-1]), H, dtype=torch.float64)
    at = [0] * N
    for pieces in ([6, 3, 8], [1, 1, 1], [1, 0, 3], [1, 1, 0]):
        idx = [int(cu[i]) + at[i] + j for i in range(N) for j in range(pieces[i])]
        r, h = (norm.forward8 if eight else norm.forward)(x[idx], res[idx], w)[0:2]
        fresh = at == [0] * N
        c = ints(np.concatenate([[0], np.cumsum(pieces)]).tolist())
        call = layer.prefill if fresh else layer.step
        got = call(r, pd["w_conv"], pd["A_log"], pd["dt_bias"], pd["w_norm"], c, cache,
                   ints([-1] * N) if fresh else slots, slots)
        Y[idx] = got
        if eight:
            unit = torch.tensor(2.0, dtype=torch.float64) ** (r.scale.cpu().double() - 127)
            rows[idx] = r.q.cpu().double() * unit.repeat_interleave(32, 1)
        else:
            rows[idx] = r.cpu().double()
        assert torch.equal(h.cpu(), (x[idx].float() + res[idx].float()).to(torch.bfloat16).cpu())
        at = [a + n for a, n in zip(at, pieces)]
    assert at == lens
    Wv = {k: v.cpu().double().numpy() for k, v in values4(layer).items()}
    prm = {k: v.double().numpy() for k, v in p.items()}
    f = oracle.proj_layer_fwd(rows.numpy(), Wv, prm, cu.astype(np.int32), HK, HV, D, D ** -0.5, round_fn=gi.round_bf16)
    assert_close("Y", host(Y), f["Y"], FWD_TOL_BF16)
    keep = cache.S()[slots.long()]
    assert_close("S", host(keep), f["S_final"], FWD_TOL_BF16)


def test_served_layer_captured():
    """Norm into 8 bits, both products and the step in one graph, replayed
    with other rows, states and slots."""
    W, p = weights(3), {k: v.to(DEV) for k, v in params(3).items()}
    layer, norm = GDNLayer4(CoreConfig(**CFG), H, W), ResidualNorm(H)
    T = 5
    cache = GDNStateCache(layer.cfg, 8)
    x, res = (torch.randn(T, H, device=DEV).to(torch.bfloat16) for _ in range(2))
    w, cu, slots = torch.randn(H, device=DEV) * 0.1, ints(list(range(T + 1))), ints([4, 1, 6, 0, 2])

    def call():
        r, h = norm.forward8(x, res, w)
        return layer.step(r, p["w_conv"], p["A_log"], p["dt_bias"], p["w_norm"], cu, cache, slots), h

    def fill():
        for k in range(1):
            cache.S(k).normal_(0, 0.1)
            cache.conv(k).normal_()

    cache.buffer.zero_()
    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        x.normal_()
        res.normal_()
        fill()
        slots.copy_(ints(np.random.default_rng(i).permutation(8)[:T].tolist()))
        start = cache.buffer.clone()
        want = [t.clone() for t in call()]
        after = cache.buffer.clone()
        cache.buffer.copy_(start)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i
        assert torch.equal(cache.buffer, after), i


def test_training_through_the_norm():
    """Norm -> layer -> residual: the gradients of x, res and the norm's
    weight against the oracle's layer and the norm's formula in 64 bits."""
    W, p = weights(4), params(4)
    pd = {k: v.to(DEV) for k, v in p.items()}
    layer, norm = GDNLayer(CoreConfig(**CFG), H, W), ResidualNorm(H)
    T = 150
    cu = np.array([0, 70, 150], dtype=np.int32)
    g = torch.Generator().manual_seed(5)
    x, res, dY, dstream = ((torch.randn(T, H, generator=g) * s).to(torch.bfloat16).to(DEV) for s in (1.0, 2.0, 1.0, 1.0))
    w = (torch.randn(H, generator=g) * 0.1).to(DEV)
    y, h = norm.forward(x, res, w)
    cud = torch.from_numpy(cu).to(DEV)
    f = layer.forward(y, pd["w_conv"], pd["A_log"], pd["dt_bias"], pd["w_norm"], cud)
    b = layer.backward(f, y, pd["w_conv"], pd["A_log"], pd["dt_bias"], pd["w_norm"], cud, dY)
    got = norm.backward(h, w, b["dX"], dstream)
    Wv = {k: v.cpu().double().numpy() for k, v in W.items()}
    prm = {k: v.double().numpy() for k, v in p.items()}
    rf = oracle.proj_layer_fwd(host(y), Wv, prm, cu, HK, HV, D, D ** -0.5, round_fn=gi.round_bf16)
    rb = oracle.proj_layer_bwd(host(y), Wv, rf, host(dY), HK, HV, D, D ** -0.5, round_fn=gi.round_bf16)
    hh, dy, ww = host(h), gi.round_bf16(rb["dX"]), host(w)
    rho = 1 / np.sqrt((hh ** 2).mean(1, keepdims=True) + 1e-6)
    n, dn = hh * rho, dy * (1 + ww)
    d = host(dstream) + rho * (dn - n * (dn * n).mean(1, keepdims=True))
    assert got["dx"] is got["dres"]
    assert_close("dx", host(got["dx"]), d, GRAD_TOL_BF16)
    assert_close("dw", host(got["dw"]), (dy * n).sum(0), GRAD_TOL_BF16)


def test_layers_agree_on_weights_that_are_in_4_bits():
    """With weights that 4 bits hold exactly the two layers differ only by the
    roundings of their products."""
    W = weights(6)
    W = {k: Linear4(v).weight(torch.bfloat16) for k, v in W.items()}
    p = {k: v.to(DEV) for k, v in params(6).items()}
    dense, four = GDNLayer(CoreConfig(**CFG), H, W), GDNLayer4(CoreConfig(**CFG), H, W)
    X = torch.randn(6, H, device=DEV).to(torch.bfloat16)
    cu, slots = ints(list(range(7))), ints([0, 1, 2, 3, 4, 5])
    out = []
    for layer in (dense, four):
        cache = GDNStateCache(layer.cfg, 6)
        out.append(layer.step(X, p["w_conv"], p["A_log"], p["dt_bias"], p["w_norm"], cu, cache, ints([-1] * 6), slots))
    assert_close("Y", host(out[1]), host(out[0]), 2 * FWD_TOL_BF16)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 3), (3, 3)])
def test_layer_of_odd_head_counts(hk, hv):
    """Columns of the joined product that do not begin at 16 bytes, rows of a
    width that is no multiple of 8: against the dense layer."""
    g = torch.Generator().manual_seed(hk + 4 * hv)
    C = 2 * hk * D + hv * D
    dims = {"x": (C, 64), "z": (hv * D, 64), "a": (hv, 64), "b": (hv, 64), "out": (64, hv * D)}
    W = {k: Linear4((torch.randn(s, generator=g) * s[1] ** -0.5).to(torch.bfloat16).to(DEV)).weight() for k, s in dims.items()}
    p = [t.to(DEV) for t in (torch.randn(C, 4, generator=g) * 0.5, torch.rand(hv, generator=g) - 2,
                             torch.randn(hv, generator=g) * 0.1, torch.randn(D, generator=g) * 0.1)]
    cfg = CoreConfig(hk=hk, hv=hv, d=D, dtype=torch.bfloat16)
    dense, four = GDNLayer(cfg, 64, W), GDNLayer4(cfg, 64, W)
    X = torch.randn(5, 64, generator=g).to(torch.bfloat16).to(DEV)
    cu = ints([0, 4, 5])
    cache = [GDNStateCache(cfg, 2) for _ in range(4)]
    want = dense.step(X, *p, cu, cache[0], ints([-1, -1]), ints([0, 1]))
    for call, c in ((four.step, cache[1]), (four.prefill, cache[2])):
        got = call(X, *p, cu, c, ints([-1, -1]), ints([0, 1]))
        assert_close("Y", host(got), host(want), 2 * FWD_TOL_BF16)
        assert_close("S", host(c.S()), host(cache[0].S()), 2 * FWD_TOL_BF16)


def test_layer_without_tokens():
    """A call of no tokens, in 16 and in 8 bits, leaves the states as they are."""
    W, p = weights(7), {k: v.to(DEV) for k, v in params(7).items()}
    layer, norm = GDNLayer4(CoreConfig(**CFG), H, W), ResidualNorm(H)
    cache = GDNStateCache(layer.cfg, 2)
    cache.buffer.fill_(7)
    before = cache.buffer.clone()
    none = torch.empty(0, H, dtype=torch.bfloat16, device=DEV)
    eight, _ = norm.forward8(none, none, torch.zeros(H, device=DEV))
    for X in (none, eight):
        for call in (layer.step, layer.prefill):
            Y = call(X, p["w_conv"], p["A_log"], p["dt_bias"], p["w_norm"], ints([0, 0]), cache, ints([1]))
            assert Y.shape == (0, H) and Y.dtype is torch.bfloat16
    assert torch.equal(cache.buffer, before)
