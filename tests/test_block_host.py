"""The operators around the core on the host (no GPU): what the C ABI and the
binding refuse before anything is launched."""
import ctypes

import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import Linear4, ResidualNorm, Rows8

P = ctypes.c_void_p(256)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(264)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
BIG = 1 << 40


def norm(**kw):
    a = dict(rows=3, n=64, dt=0, rt=0, x=P, ldx=64, res=P, ldr=64, w=P, eps=1e-6, h=P, ldh=64, y=P, ldy=64)
    a.update(kw)
    return L.load().gdn_add_norm_fwd(*a.values(), None)


def norm8(**kw):
    a = dict(rows=3, n=64, dt=0, rt=0, x=P, ldx=64, res=P, ldr=64, w=P, eps=1e-6, h=P, ldh=64, q=P, ldq=64, s=P,
             lds=2)
    a.update(kw)
    return L.load().gdn_add_norm_fwd_mx8(*a.values(), None)


def back(**kw):
    a = dict(rows=3, n=64, dt=0, rt=1, h=P, ldh=64, w=P, eps=1e-6, dy=P, lddy=64, dh=P, lddh=64, dx=P, lddx=64,
             dres=P, lddr=64, dw=P, ws=P, ws_bytes=BIG)
    a.update(kw)
    return L.load().gdn_add_norm_bwd(*a.values(), None)


SHAPES = [(dict(rows=-1), INVALID), (dict(n=0), INVALID), (dict(n=12), UNSUPPORTED), (dict(n=16392, ldx=16392),
          UNSUPPORTED), (dict(dt=3), INVALID), (dict(rt=7), INVALID), (dict(dt=1, rt=0), UNSUPPORTED),
          (dict(dt=0, rt=2), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
          (dict(w=None), INVALID), (dict(w=ODD), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=ODD), ALIGNMENT), (dict(res=ODD), ALIGNMENT),
    (dict(h=ODD), ALIGNMENT), (dict(y=ODD), ALIGNMENT), (dict(ldx=56), INVALID), (dict(ldx=68), ALIGNMENT),
    (dict(ldr=56), INVALID), (dict(ldh=68), ALIGNMENT), (dict(ldy=56), INVALID),
    (dict(rows=0, x=None, res=None, h=None, y=None), OK)])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(lds=1), INVALID),
    (dict(n=40), UNSUPPORTED), (dict(ldq=72), ALIGNMENT), (dict(ldq=48), INVALID), (dict(q=ODD), ALIGNMENT),
    (dict(rows=0, x=None, res=None, h=None, q=None, s=None), OK)])
def test_norm8_refusals(kw, status):
    assert norm8(**kw) == status


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(h=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None, dres=None, dw=None), INVALID),
    (dict(h=ODD), ALIGNMENT), (dict(dy=ODD), ALIGNMENT), (dict(dh=ODD), ALIGNMENT), (dict(dx=ODD), ALIGNMENT),
    (dict(dres=ODD), ALIGNMENT), (dict(dw=ODD), ALIGNMENT), (dict(ldh=56), INVALID), (dict(lddy=68), ALIGNMENT),
    (dict(lddh=56), INVALID), (dict(lddx=56), INVALID), (dict(lddr=68), ALIGNMENT), (dict(ws=None), WORKSPACE),
    (dict(ws=ODD), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(rows=0, h=None, dy=None, w=None), INVALID),
    (dict(rows=0, h=None, dy=None, dx=None, dres=None, dw=None), OK)])
def test_norm_backward_refusals(kw, status):
    assert back(**kw) == status


def test_norm_backward_workspace():
    f = L.gdn_add_norm_bwd_workspace
    assert f(-1, 64) == 0 and f(3, 0) == 0 and f(3, 16392) == 0
    assert f(1, 64) >= 4 * 64 and f(1 << 40, 16384) <= 1 << 30
    assert all(f(a, 2560) <= f(b, 2560) for a, b in zip((0, 1, 5, 100, 5000), (1, 5, 100, 5000, 100000)))


@pytest.mark.parametrize("n,k", [(0, 64), (8, 0), (-1, 64), (8, 16), (8, 48), ((1 << 22) + 1, 32), (8, (1 << 20) + 32),
                                 (1 << 22, 1 << 20)])
def test_no_weights_of_such_sizes(n, k):
    lib = L.load()
    st = INVALID if n < 1 or k < 1 else UNSUPPORTED
    assert L.gdn_w4_bytes(n, k) == 0
    assert lib.gdn_w4_pack(n, k, 0, P, 1 << 21, P, BIG, None) == st
    assert lib.gdn_w4_arrange(n, k, P, 1 << 21, P, 1 << 21, P, BIG, None) == st
    assert lib.gdn_w4_unpack(n, k, P, BIG, 0, P, 1 << 21, None) == st
    assert lib.gdn_w4_fwd(1, n, k, 0, P, 1 << 21, P, BIG, P, 1 << 23, None) == st
    assert lib.gdn_w4_fwd_mx8(1, n, k, P, 1 << 21, P, 1 << 21, P, BIG, 0, P, 1 << 23, None) == st
    with pytest.raises(ValueError):
        L.W4(torch.empty(64, dtype=torch.uint8), n, k)


def test_packed_bytes_cover_codes_and_scales():
    for n, k in ((1, 32), (16, 512), (17, 544), (2560, 6144)):
        pad = -(-n // 16) * 16 * -(-k // 512) * 512
        assert L.gdn_w4_bytes(n, k) == pad // 2 + pad // 32


@pytest.mark.parametrize("kw,status", [
    (dict(dt=5), INVALID), (dict(w=None), INVALID), (dict(w=ODD), ALIGNMENT), (dict(ldw=56), INVALID),
    (dict(ldw=68), ALIGNMENT), (dict(packed=None), INVALID), (dict(packed=ODD), ALIGNMENT), (dict(size=4351), INVALID)])
def test_pack_and_unpack_refusals(kw, status):
    a = dict(dt=0, w=P, ldw=64, packed=P, size=4352)
    a.update(kw)
    lib = L.load()
    assert lib.gdn_w4_pack(8, 64, a["dt"], a["w"], a["ldw"], a["packed"], a["size"], None) == status
    assert lib.gdn_w4_unpack(8, 64, a["packed"], a["size"], a["dt"], a["w"], a["ldw"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(c=None), INVALID), (dict(c=ODD), ALIGNMENT), (dict(ldc=16), INVALID), (dict(ldc=40), ALIGNMENT),
    (dict(s=None), INVALID), (dict(lds=1), INVALID), (dict(packed=None), INVALID), (dict(size=4351), INVALID)])
def test_arrange_refusals(kw, status):
    a = dict(c=P, ldc=32, s=P, lds=2, packed=P, size=4352)
    a.update(kw)
    assert L.load().gdn_w4_arrange(8, 64, *a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(dt=3), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(x=ODD), ALIGNMENT), (dict(y=ODD), ALIGNMENT), (dict(ldx=56), INVALID), (dict(ldx=68), ALIGNMENT),
    (dict(ldy=8), INVALID), (dict(ldy=20), ALIGNMENT), (dict(packed=None), INVALID), (dict(size=4351), INVALID),
    (dict(rows=0, x=None, y=None), OK)])
def test_product_refusals(kw, status):
    a = dict(rows=2, dt=0, x=P, ldx=64, packed=P, size=4352, y=P, ldy=16)
    a.update(kw)
    lib = L.load()
    assert lib.gdn_w4_fwd(a["rows"], 10, 64, a["dt"], a["x"], a["ldx"], a["packed"], a["size"], a["y"], a["ldy"],
                          None) == status
    if a["ldx"] != 68:       # rows of 8 bits: see below
        assert lib.gdn_w4_fwd_mx8(a["rows"], 10, 64, a["x"], a["ldx"], P, 2, a["packed"], a["size"], a["dt"], a["y"],
                                  a["ldy"], None) == status


def test_product_of_8_bit_rows_refusals():
    f = L.load().gdn_w4_fwd_mx8
    assert f(2, 10, 64, P, 72, P, 2, P, 4352, 0, P, 16, None) == ALIGNMENT
    assert f(2, 10, 64, P, 64, None, 2, P, 4352, 0, P, 16, None) == INVALID
    assert f(2, 10, 64, P, 64, P, 1, P, 4352, 0, P, 16, None) == INVALID


def test_binding_refuses_before_the_call():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros(3, 64, dtype=bf), torch.zeros(64)
    norm = ResidualNorm(64, device="cpu")
    with pytest.raises(ValueError, match="host tensor"):
        norm.forward(x, x, w)
    with pytest.raises(TypeError):
        norm.forward(x, x.float(), w)                       # the stream is bf16 here
    with pytest.raises(ValueError):
        norm.forward(x.float(), x, w)
    with pytest.raises(ValueError):
        norm.forward(x[:, :32], x[:, :32], w[:32])
    with pytest.raises(ValueError):
        norm.forward(x, x[:2], w)
    with pytest.raises(TypeError):
        norm.forward(x, x, w.to(bf))
    with pytest.raises(ValueError):
        norm.forward(x, x, w[:32])
    with pytest.raises(ValueError):
        norm.forward(x.t().contiguous().t(), x, w)          # columns are not adjacent
    with pytest.raises(TypeError):
        norm.backward(x.float(), w, x)
    with pytest.raises(ValueError):
        norm.backward(x, w, x[:2])
    with pytest.raises(ValueError):
        norm.backward(x, w, x, x[:, :32])
    with pytest.raises(TypeError):
        ResidualNorm(64, dtype=f32, res_dtype=bf, device="cpu")
    with pytest.raises(ValueError):
        ResidualNorm(60, device="cpu")
    with pytest.raises(ValueError, match="host tensor"):
        Linear4(torch.zeros(8, 64, dtype=bf))
    with pytest.raises(ValueError):
        Linear4(torch.zeros(8, 48, dtype=bf))
    with pytest.raises(TypeError):
        Linear4(torch.zeros(8, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        Linear4.from_codes(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        Linear4.from_codes(torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8, 2, dtype=torch.uint8))
    proj = Linear4.__new__(Linear4)
    proj._make(8, 64, torch.zeros(1))
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(3, 2, dtype=torch.uint8)
    for bad in (x[:, :32], torch.zeros(3, 64, dtype=torch.float64), Rows8(q[:, :32], s[:, :1])):
        with pytest.raises((ValueError, TypeError)):
            proj(bad)
    for bad in ((x, s), (q, s[:, :1]), (q, s.to(torch.int8)), (q[:, :40], s), (q.t().contiguous().t(), s), (q[0], s),
                (q, s, torch.int8)):
        with pytest.raises((ValueError, TypeError)):
            Rows8(*bad)
    with pytest.raises(ValueError, match="host tensor"):
        norm.forward8(x, x, w)
    with pytest.raises(ValueError, match="host tensor"):
        proj(Rows8(q, s))
    with pytest.raises(ValueError, match="host tensor"):
        proj(x)
