"""The residual norm over rows enough for every workgroup to take several,
at widths from 520 to 16384: every row against the formula in 64 bits, and bit by
bit against calls of fewer rows, which take other variants or other turns.
Tolerances as in test_gpu_add_norm; dw is in test_add_norm_dw."""
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import ResidualNorm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
EPS = 1e-5
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def make(T, n, dt, rt, pad=0):
    g = torch.Generator(device=DEV).manual_seed(T + n)

    def rows(to, std):
        t = torch.full((T + 2, n + pad), 7.0, dtype=DT[to], device=DEV)
        t[1:-1, :n] = torch.randn(T, n, generator=g, device=DEV) * std
        return t

    d = {k: rows(to, std) for k, to, std in (("x", dt, 1.0), ("res", rt, 3.0), ("dy", dt, 0.5), ("dh", rt, 0.5))}
    d["w"] = torch.randn(n, generator=g, device=DEV) * 0.3
    return d


def inner(t, n):
    return t[1:-1, :n]


def kept(t, n):
    """The bands around the rows."""
    return (t[0] == 7).all() and (t[-1] == 7).all() and (t[:, n:] == 7).all()


def near(got, ref, tol, what):
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), \
        f"{what}: off by {float((off / tol.clamp(min=1e-300)).max()):.3g} of what it may be"


def fwd(x, res, w):
    h = x.double() + res.double()
    return h, h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * (1 + w.double())


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n,pad", [(2309, 520, 8), (4099, 4096, 0), (2309, 4128, 24), (2057, 8192, 0), (2051, 8200, 8),
                                     (2053, 16384, 0)])
def test_forward(T, n, pad, dt, rt):
    d = make(T, n, dt, rt, pad)
    x, res = inner(d["x"], n), inner(d["res"], n)
    hr, yr = fwd(x, res, d["w"])
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    y, h = norm.forward(x, res, d["w"])
    near(h, hr, (half(DT[rt]) + U) * hr.abs() + tiny(DT[rt]), "h")
    near(y, yr, (half(DT[dt]) + 48 * U) * yr.abs() + tiny(DT[dt]), "y")
    for a in (0, 1000, T - 333):
        s = slice(a, a + 333)
        y1, h1 = norm.forward(x[s], res[s], d["w"])
        assert torch.equal(y1, y[s]) and torch.equal(h1, h[s])
    L.gdn_add_norm_fwd(x, res, d["w"], res, x, EPS)        # in place, between bands
    assert torch.equal(x, y) and torch.equal(res, h)
    assert kept(d["x"], n) and kept(d["res"], n)


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n", [(2309, 544), (2309, 2592), (4099, 4096), (2057, 4128), (2057, 8192), (2053, 16384)])
def test_forward_into_8_bits(T, n, dt, rt):
    """The scales are the smallest that hold their groups, values are within
    half a step of e4m3 (2^-4 of themselves, 2^-10 of the scale below its
    normal numbers)."""
    d = make(T, n, dt, rt)
    d["x"][5], d["res"][5] = 0, 0
    x, res = inner(d["x"], n), inner(d["res"], n)
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    rows, h = norm.forward8(x, res, d["w"])
    assert torch.equal(h, norm.forward(x, res, d["w"])[1])
    _, yr = fwd(x, res, d["w"])
    amax = yr.view(T, -1, 32).abs().amax(2)
    unit = torch.exp2(rows.scale.double() - 127)
    assert (amax <= 448 * unit * (1 + 48 * U)).all()
    assert ((amax > 224 * unit * (1 - 48 * U)) | (rows.scale == 0)).all()
    assert (rows.scale[4] == 0).all() and (rows.q[4].float() == 0).all()
    wide = unit.repeat_interleave(32, 1)
    near(rows.q.float().double() * wide, yr,
         torch.maximum(yr.abs() * 2.0 ** -4, wide * 2.0 ** -10) + 48 * U * yr.abs(), "values")
    for a in (0, 1000, T - 333):
        s = slice(a, a + 333)
        r1, _ = norm.forward8(x[s], res[s], d["w"])
        assert torch.equal(r1.q.view(torch.uint8), rows.q[s].view(torch.uint8)) and torch.equal(r1.scale, rows.scale[s])
    q = torch.full((T + 2, n + 16), 1.0, device=DEV).to(torch.float8_e4m3fn)
    scale = torch.full((T + 2, n // 32 + 3), 7, dtype=torch.uint8, device=DEV)
    L.gdn_add_norm_fwd_mx8(x, res, d["w"], None, q[1:-1, :n], scale[1:-1, 1:-2], EPS)
    assert torch.equal(q[1:-1, :n].view(torch.uint8), rows.q.view(torch.uint8))
    assert torch.equal(scale[1:-1, 1:-2], rows.scale)
    edge = q.float()
    assert (edge[0] == 1).all() and (edge[-1] == 1).all() and (edge[:, n:] == 1).all()
    assert (scale[0] == 7).all() and (scale[-1] == 7).all() and (scale[:, 0] == 7).all() and (scale[:, -2:] == 7).all()


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n,pad", [(3001, 520, 8), (2309, 4096, 0), (2309, 4128, 24), (1031, 8192, 0), (777, 8200, 8),
                                     (523, 16384, 0)])
def test_backward(T, n, pad, dt, rt):
    d = make(T, n, dt, rt, pad)
    h, dy, dh, w = inner(d["res"], n), inner(d["dy"], n), inner(d["dh"], n), d["w"]
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    g = norm.backward(h, w, dy, dh)
    hd, wy = h.double(), dy.double() * (1 + w.double())
    rho = (hd.square().mean(1, keepdim=True) + EPS).rsqrt()
    v = hd * rho
    ref = dh.double() + rho * (wy - v * (wy * v).mean(1, keepdim=True))
    size = dh.double().abs() + rho * (wy.abs() + v.abs() * (wy * v).abs().mean(1, keepdim=True))
    for k in ("dx", "dres"):
        t = g[k].dtype
        near(g[k], ref, half(t) * ref.abs() + 128 * U * size + tiny(t), k)
    for a in (0, 200, T - 77):
        s = slice(a, a + 77)
        g1 = norm.backward(h[s], w, dy[s], dh[s])
        assert torch.equal(g1["dx"], g["dx"][s]) and torch.equal(g1["dres"], g["dres"][s])
    without = norm.backward(h, w, dy)["dres"]
    near(without, ref - dh.double(), half(without.dtype) * (ref - dh.double()).abs() + 128 * U * size
         + tiny(without.dtype), "dres without dh")
    dw = torch.empty(n, device=DEV)
    ws = torch.empty(L.gdn_add_norm_bwd_workspace(T, n), dtype=torch.uint8, device=DEV)
    L.gdn_add_norm_bwd(h, w, dy, dh, dy, dh, dw, ws, EPS)       # in place, between bands
    assert torch.equal(dy, g["dx"]) and torch.equal(dh, g["dres"]) and torch.equal(dw, g["dw"])
    assert kept(d["dy"], n) and kept(d["dh"], n)
