"""The residual norm against the formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and e = half a step of the
storage type (torch.finfo(t).eps / 2):

forward   y = v rho (1 + w).  A thread adds at most 40 squares, the rest is a
          tree: the sum of n <= 16384 positive terms is within 40 + 6 + 16 + 4
          = 66 u of itself, rho within half of that, 33 u, and a few u of the
          quotient, the root (2 u) and three products: 48 u in all, and e.
backward  d = dh + rho (dn - n m): every term carries at most 48 u as above, m
          66 u of mean |dn n| more: 128 u of |dh| + rho (|dn| + |n| mean |dn n|),
          and e of d.
dw        a sum over T rows in some order: (T + 48) u of sum |dy n|.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import ResidualNorm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = [(1, 8), (1, 2560), (2, 512), (3, 520), (5, 1024), (4, 1032), (7, 2552), (6, 2568), (9, 4096), (3, 8192),
         (2, 8200), (3, 16384), (333, 64), (70, 1000)]
EPS = 1e-5


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half a step of the type's smallest values."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def make(T, n, dt, rt, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + n)

    def rows(to, std):
        t = torch.full((T, n + pad), float("nan")).to(to)
        t[:, :n] = torch.randn(T, n, generator=g).mul(std).to(to)
        return t.to(DEV)[:, :n]

    return dict(x=rows(dt, 1.0), res=rows(rt, 3.0), w=(torch.randn(n, generator=g) * 0.3).to(DEV), dy=rows(dt, 0.5),
                dh=rows(rt, 0.5))


def ref_fwd(x, res, w, eps=EPS):
    h = x.cpu().double() + (res.cpu().double() if res is not None else 0)
    return h, h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * (1 + w.cpu().double())


def near(got, ref, tol, what):
    got = got.cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), \
        f"{what}: off by {float((off / tol.clamp(min=1e-300)).max()):.3g} of what it may be"


def check_fwd(y, h, d, rt, eps=EPS, res=True):
    dt = y.dtype
    hr, yr = ref_fwd(d["x"], d["res"] if res else None, d["w"], eps)
    near(h, hr, (half(rt) + U) * hr.abs() + tiny(rt), "h")
    near(y, yr, (half(dt) + 48 * U) * yr.abs() + tiny(dt), "y")


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n", SIZES)
def test_forward(T, n, dt, rt):
    d = make(T, n, DT[dt], DT[rt])
    y, h = ResidualNorm(n, DT[dt], DT[rt], EPS).forward(d["x"], d["res"], d["w"])
    assert y.dtype == DT[dt] and h.dtype == DT[rt]
    check_fwd(y, h, d, DT[rt])


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n", SIZES)
def test_backward(T, n, dt, rt):
    d = make(T, n, DT[dt], DT[rt], 1)
    for dh in (d["dh"], None):
        g = ResidualNorm(n, DT[dt], DT[rt], EPS).backward(d["res"], d["w"], d["dy"], dh)
        check_bwd(g, d["res"], d["w"], d["dy"], dh)


def check_bwd(g, h, w, dy, dh, eps=EPS):
    h, w, dy = h.cpu().double(), w.cpu().double(), dy.cpu().double()
    T = h.shape[0]
    up = torch.zeros_like(h) if dh is None else dh.cpu().double()
    rho = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    n, dn = h * rho, dy * (1 + w)
    ref = up + rho * (dn - n * (dn * n).mean(1, keepdim=True))
    size = up.abs() + rho * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    for k in ("dx", "dres"):
        t = g[k].dtype
        near(g[k], ref, half(t) * ref.abs() + 128 * U * size + tiny(t), k)
    near(g["dw"], (dy * n).sum(0), (T + 48) * U * (dy * n).abs().sum(0) + 1e-300, "dw")


@pytest.mark.parametrize("dt,rt", TYPES)
def test_gradients_agree_with_differences(dt, rt):
    """The directional derivative of sum(dy y) + sum(dh h), formed in 64 bits
    from the definition, against the kernel's gradients."""
    T, n = 4, 264
    d = make(T, n, DT[dt], DT[rt], 2)
    g = ResidualNorm(n, DT[dt], DT[rt], EPS).backward(d["res"], d["w"], d["dy"], d["dh"])
    gen = torch.Generator().manual_seed(3)
    h, w, dy, dh = (d[k].cpu().double() for k in ("res", "w", "dy", "dh"))
    for k in range(4):
        uh, uw = torch.randn(T, n, generator=gen).double(), torch.randn(n, generator=gen).double()

        def loss(s):
            hh, ww = h + s * uh, w + s * uw
            return ((hh * (hh.square().mean(1, keepdim=True) + EPS).rsqrt() * (1 + ww)) * dy).sum() + (hh * dh).sum()

        step = 1e-4
        want = (loss(step) - loss(-step)) / (2 * step)
        rows, dw = g["dres"].cpu().double(), g["dw"].cpu().double()
        got = (rows * uh).sum() + (dw * uw).sum()
        # the gradients' own roundings, and step^2 / 6 of third derivatives of order one a value
        tol = ((half(DT[rt]) + 200 * U) * (rows.abs() * uh.abs()).sum() + 200 * U * (dw.abs() * uw.abs()).sum()
               + step ** 2 * T * n * 10)
        assert abs(got - want) <= tol, (float(got), float(want), float(tol))


@pytest.mark.parametrize("dt,rt", TYPES)
def test_rows_of_wider_buffers(dt, rt):
    """Strided rows; what lies between them is neither read (NaN) nor written."""
    T, n, pad = 37, 1000, 24
    d = make(T, n, DT[dt], DT[rt], 3, pad)
    y0 = torch.full((T + 2, n + pad), 7.0, dtype=DT[dt], device=DEV)
    h0 = torch.full((T + 2, n + pad), 7.0, dtype=DT[rt], device=DEV)
    y, h = y0[1:-1, :n], h0[1:-1, :n]
    L.gdn_add_norm_fwd(d["x"], d["res"], d["w"], h, y, EPS)
    check_fwd(y, h, d, DT[rt])
    dx0, dr0 = torch.full_like(y0, 7.0), torch.full_like(h0, 7.0)
    dx, dr, dw = dx0[1:-1, :n], dr0[1:-1, :n], torch.empty(n, device=DEV)
    ws = torch.empty(L.gdn_add_norm_bwd_workspace(T, n), dtype=torch.uint8, device=DEV)
    L.gdn_add_norm_bwd(d["res"], d["w"], d["dy"], d["dh"], dx, dr, dw, ws, EPS)
    check_bwd({"dx": dx, "dres": dr, "dw": dw}, d["res"], d["w"], d["dy"], d["dh"])
    for t in (y0, h0, dx0, dr0):
        assert (t[0] == 7).all() and (t[-1] == 7).all() and (t[:, n:] == 7).all()


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("n", [64, 2560, 6144, 16384])
def test_in_place(n, dt, rt):
    T = 9
    d = make(T, n, DT[dt], DT[rt], 4)
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    y, h = norm.forward(d["x"], d["res"], d["w"])
    x2, r2 = d["x"].clone(), d["res"].clone()
    L.gdn_add_norm_fwd(x2, r2, d["w"], r2, x2, EPS)        # h over res, y over x
    assert torch.equal(x2, y) and torch.equal(r2, h)
    g = norm.backward(h, d["w"], d["dy"], d["dh"])
    dx2, dr2 = d["dy"].clone(), d["dh"].clone()
    L.gdn_add_norm_bwd(h, d["w"], dx2, dr2, dx2, dr2, None, None, EPS)
    assert torch.equal(dx2, g["dx"]) and torch.equal(dr2, g["dres"])


@pytest.mark.parametrize("dt,rt", TYPES)
def test_without_residual_and_outputs_left_out(dt, rt):
    T, n = 11, 640
    d = make(T, n, DT[dt], DT[rt], 5)
    y, h = ResidualNorm(n, DT[dt], DT[rt], EPS).forward(d["x"], None, d["w"])
    check_fwd(y, h, d, DT[rt], res=False)
    if dt == rt:
        assert h is d["x"]
    full = ResidualNorm(n, DT[dt], DT[rt], EPS).forward(d["x"], d["res"], d["w"])
    y2 = torch.empty_like(y)
    L.gdn_add_norm_fwd(d["x"], d["res"], d["w"], None, y2, EPS)
    assert torch.equal(y2, full[0])
    g = ResidualNorm(n, DT[dt], DT[rt], EPS).backward(d["res"], d["w"], d["dy"], d["dh"])
    ws = torch.empty(L.gdn_add_norm_bwd_workspace(T, n), dtype=torch.uint8, device=DEV)
    one = {"dx": torch.empty_like(d["dy"]), "dres": torch.empty_like(d["dh"]), "dw": torch.empty(n, device=DEV)}
    for k in one:
        out = [one[m] if m == k else None for m in ("dx", "dres", "dw")]
        L.gdn_add_norm_bwd(d["res"], d["w"], d["dy"], d["dh"], *out, ws if k == "dw" else None, EPS)
        assert torch.equal(one[k], g[k]), k


def test_no_rows():
    for rt in (torch.bfloat16, torch.float32):
        norm = ResidualNorm(64, torch.bfloat16, rt)
        x, r, w = (torch.empty(0, 64, dtype=t, device=DEV) for t in (torch.bfloat16, rt, rt))
        w = torch.zeros(64, device=DEV)
        y, h = norm.forward(x, r, w)
        rows, _ = norm.forward8(x, r, w)
        assert y.shape == h.shape == rows.q.shape == (0, 64) and rows.scale.shape == (0, 2)
        g = norm.backward(h, w, y, r)
        assert g["dx"].shape == (0, 64) and (g["dw"] == 0).all()


@pytest.mark.parametrize("dt,rt", TYPES)
def test_values_at_the_edges(dt, rt):
    """Rows of zeros; NaN and infinities stay in their row; large values do
    not overflow in fp32 where their squares fit; tiny ones keep eps."""
    n = 1040
    d = make(6, n, DT[dt], DT[rt], 6)
    d["x"][0], d["res"][0] = 0, 0
    d["x"][1, 5] = float("nan")
    d["x"][2, 7] = float("inf")
    d["res"][3, 9] = -float("inf")
    d["x"][4] = 3e4
    d["x"][5], d["res"][5] = 1e-6, 0
    y, h = ResidualNorm(n, DT[dt], DT[rt], EPS).forward(d["x"], d["res"], d["w"])
    assert (y[0] == 0).all() and (h[0] == 0).all()
    assert y[1].isnan().all() and torch.isnan(h[1, 5]) and h[1, :5].isfinite().all()
    assert torch.isinf(h[2, 7]) and torch.isinf(h[3, 9])
    keep = [0, 4, 5]
    part = {k: d[k][keep] if d[k].dim() == 2 else d[k] for k in d}
    hr, yr = ref_fwd(part["x"], part["res"], part["w"])
    near(y[keep], yr, (half(DT[dt]) + 48 * U) * yr.abs() + tiny(DT[dt]), "y")
    clean = make(6, n, DT[dt], DT[rt], 6)
    g = ResidualNorm(n, DT[dt], DT[rt], EPS).backward(h[keep].contiguous(), d["w"], clean["dy"][keep].contiguous())
    check_bwd(g, h[keep], d["w"], clean["dy"][keep], None)


@pytest.mark.parametrize("n", [64, 2560, 8192, 16384])
def test_repeats_bit_by_bit_and_rows_alone(n):
    """A row's values do not depend on the batch it is in; dw does not change
    from run to run."""
    T = 77
    d = make(T, n, torch.bfloat16, torch.float32, 7)
    norm = ResidualNorm(n, torch.bfloat16, torch.float32, EPS)
    y, h = norm.forward(d["x"], d["res"], d["w"])
    g = norm.backward(h, d["w"], d["dy"], d["dh"])
    for _ in range(3):
        assert torch.equal(norm.forward(d["x"], d["res"], d["w"])[0], y)
        again = norm.backward(h, d["w"], d["dy"], d["dh"])
        assert all(torch.equal(again[k], g[k]) for k in g)
    y1, h1 = norm.forward(d["x"][40:41], d["res"][40:41], d["w"])
    assert torch.equal(y1[0], y[40]) and torch.equal(h1[0], h[40])


@pytest.mark.parametrize("T,n,dt,rt", [(20000, 256, "bf16", "bf16"), (9000, 2560, "bf16", "fp32"),
                                       (5000, 3200, "fp16", "fp16")])
def test_many_rows(T, n, dt, rt):
    d = make(T, n, DT[dt], DT[rt], 8)
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    y, h = norm.forward(d["x"], d["res"], d["w"])
    check_fwd(y, h, d, DT[rt])
    check_bwd(norm.backward(h, d["w"], d["dy"], d["dh"]), h, d["w"], d["dy"], d["dh"])


@pytest.mark.parametrize("T,n,dt,rt", [(349601, 72, "fp32", "fp32"), (95407, 264, "fp32", "fp32"), (70001, 480, "bf16", "fp32"),
                                       (105003, 512, "fp16", "fp16"), (211003, 256, "bf16", "bf16")])
def test_narrow_rows_beyond_the_cache(T, n, dt, rt):
    """The last rows against 64 bits, all of them against calls of fewer rows
    bit by bit (in 8 bits as well), dw against 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(n)
    x, res, up = (torch.randn(T, n, generator=g, device=DEV) for _ in range(3))
    x, res, up, dy = x.to(DT[dt]), (res * 3).to(DT[rt]), up.to(DT[rt]), (up * 2).to(DT[dt])
    w = torch.randn(n, generator=g, device=DEV) * 0.1
    norm = ResidualNorm(n, DT[dt], DT[rt], EPS)
    y, h = norm.forward(x, res, w)
    b = norm.backward(h, w, dy, up)
    eight = norm.forward8(x, res, w)[0] if n % 32 == 0 else None
    for at in (0, T - 20000):
        s = slice(at, at + 20000)
        y1, h1 = norm.forward(x[s], res[s], w)
        b1 = norm.backward(h1, w, dy[s], up[s])
        assert torch.equal(y[s], y1) and torch.equal(h[s], h1)
        assert torch.equal(b["dx"][s], b1["dx"]) and torch.equal(b["dres"][s], b1["dres"])
        if eight is not None:
            e1 = norm.forward8(x[s], res[s], w)[0]
            assert torch.equal(eight.q[s].view(torch.uint8), e1.q.view(torch.uint8)) and torch.equal(eight.scale[s], e1.scale)
    s = slice(T - 500, T)
    check_fwd(y[s], h[s], {"x": x[s], "res": res[s], "w": w}, DT[rt])
    hd, dyd = h.double(), dy.double()
    t = dyd * hd * (hd.square().mean(1, keepdim=True) + EPS).rsqrt()
    near(b["dw"], t.sum(0).cpu(), ((T + 48) * U * t.abs().sum(0) + 1e-300).cpu(), "dw")


def test_more_rows_than_a_launch_and_offsets_beyond_32_bits():
    """2^22 + 3 rows: more than a launch's workgroups, and elements beyond
    2^32; rows here and there against the formula."""
    T, n = (1 << 22) + 3, 1032
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, 1 << 20):
        x[a:a + (1 << 20)].normal_(generator=g)
    w = torch.randn(n, generator=g, device=DEV) * 0.3
    norm = ResidualNorm(n, eps=EPS)
    y, h = norm.forward(x, x, w)
    at = [0, 1, 2, 77, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 2, (1 << 22) - 1, 1 << 22, T - 2, T - 1]
    part = {"x": x[at], "res": x[at], "w": w}
    check_fwd(y[at], h[at], part, torch.bfloat16)
    del y
    g2 = norm.backward(h, w, x, x)
    one = norm.backward(h[at], w, x[at], x[at])
    assert torch.equal(g2["dx"][at], one["dx"])
    assert torch.isfinite(g2["dw"]).all()


# ------------------------------------------------------------------ 8 bits
def values8(rows):
    """The values that 8-bit rows stand for, in 64 bits."""
    unit = torch.tensor(2.0, dtype=torch.float64) ** (rows.scale.cpu().double() - 127)
    return rows.q.cpu().double() * unit.repeat_interleave(32, 1)


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n", [(1, 32), (1, 2560), (3, 544), (5, 1056), (6, 2592), (2, 8192), (2, 16384), (200, 64)])
def test_forward8(T, n, dt, rt):
    """Scales are the smallest that hold the group (48 u of its largest
    decide either way at the border); values are within half a step: 2^-4 of
    themselves, or 2^-10 of the scale below its smallest normal value."""
    d = make(T, n, DT[dt], DT[rt], 9)
    d["x"][0, :32], d["res"][0, :32] = 0, 0
    rows, h = ResidualNorm(n, DT[dt], DT[rt], EPS).forward8(d["x"], d["res"], d["w"])
    assert rows.dtype == DT[dt] and rows.q.dtype == torch.float8_e4m3fn and rows.scale.shape == (T, n // 32)
    y, h2 = ResidualNorm(n, DT[dt], DT[rt], EPS).forward(d["x"], d["res"], d["w"])
    assert torch.equal(h, h2)
    _, yr = ref_fwd(d["x"], d["res"], d["w"])
    amax = yr.view(T, -1, 32).abs().amax(2)
    unit = torch.tensor(2.0, dtype=torch.float64) ** (rows.scale.cpu().double() - 127)
    assert (amax <= 448 * unit * (1 + 48 * U)).all()
    assert ((amax > 224 * unit * (1 - 48 * U)) | (rows.scale.cpu() == 0)).all()
    assert rows.scale[0, 0] == 0 and (rows.q[0, :32].float() == 0).all()
    near(values8(rows), yr, torch.maximum(yr.abs() * 2.0 ** -4, unit.repeat_interleave(32, 1) * 2.0 ** -10)
         + 48 * U * yr.abs(), "values")


def test_forward8_ties_and_edges():
    """Values that fall on the format's ties and borders, exactly: rows whose
    mean square is one give y = h (eps = 0)."""
    n = 64
    a = torch.zeros(3, n, dtype=torch.float64)
    # a row of ones: amax 1 = 256 * 2^-8 -> scale 2^-8, q = 256
    a[0] = 1
    # mean square one with a spread: 32 values of a, 32 of b, a^2 + b^2 = 2
    a[1, :32], a[1, 32:] = 1.4, (2 - 1.96) ** 0.5
    a[2, 0] = 8                                      # 64 / 64: the rest zeros
    x = a.float().to(DEV)
    w = torch.zeros(n, device=DEV)
    rows, _ = ResidualNorm(n, torch.float32, eps=0.0).forward8(x, None, w)
    assert (rows.scale[0] == 127 - 8).all() and (rows.q[0].float() == 256).all()
    assert rows.scale[2].tolist() == [127 - 5, 0] and rows.q[2, 0].float() == 256
    assert (rows.q[2, 1:].float() == 0).all()
    near(values8(rows)[1:2], a[1:2], a[1:2].abs() * (2.0 ** -4 + 48 * U), "spread")
    x[1, 3], x[2, 40] = float("nan"), float("inf")
    rows, _ = ResidualNorm(n, torch.float32, eps=0.0).forward8(x, None, w)
    assert (rows.q[0].float() == 256).all()
    assert rows.q[1].float().isnan().all()           # NaN in a row: rho is NaN
    assert rows.q[2, 40].float().isnan()             # inf * 0


def test_forward8_rows_of_wider_buffers():
    T, n = 19, 96
    d = make(T, n, torch.bfloat16, torch.bfloat16, 10, 8)
    want, _ = ResidualNorm(n).forward8(d["x"], d["res"], d["w"])
    q0 = torch.full((T + 2, n + 16), 1.0, device=DEV).to(torch.float8_e4m3fn)
    s0 = torch.full((T + 2, 7), 9, dtype=torch.uint8, device=DEV)
    L.gdn_add_norm_fwd_mx8(d["x"], d["res"], d["w"], None, q0[1:-1, :n], s0[1:-1, 2:5])
    assert torch.equal(q0[1:-1, :n].view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(s0[1:-1, 2:5], want.scale)
    q = q0.float()
    assert (q[0] == 1).all() and (q[-1] == 1).all() and (q[:, n:] == 1).all()
    assert (s0[0] == 9).all() and (s0[-1] == 9).all() and (s0[:, :2] == 9).all() and (s0[:, 5:] == 9).all()


# ------------------------------------------------------------------ streams and graphs
def test_other_streams_and_two_at_once():
    T, n = 3000, 2560
    ds = [make(T, n, torch.bfloat16, torch.bfloat16, s) for s in (11, 12)]
    norm = ResidualNorm(n, eps=EPS)
    want = [(norm.forward(d["x"], d["res"], d["w"]), norm.backward(d["res"], d["w"], d["dy"], d["dh"])) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [None, None]
        for i, d in enumerate(ds):
            with torch.cuda.stream(streams[i]):
                got[i] = (norm.forward(d["x"], d["res"], d["w"]), norm.backward(d["res"], d["w"], d["dy"], d["dh"]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0][0], b[0][0]) and torch.equal(a[0][1], b[0][1])
            assert all(torch.equal(a[1][k], b[1][k]) for k in b[1])


def test_captured_and_replayed():
    T, n = 50, 2560
    d = make(T, n, torch.bfloat16, torch.float32, 13)
    norm = ResidualNorm(n, torch.bfloat16, torch.float32, EPS)

    def call():
        y, h = norm.forward(d["x"], d["res"], d["w"])
        rows, _ = norm.forward8(d["x"], d["res"], d["w"])
        g = norm.backward(h, d["w"], d["dy"], d["dh"])
        return [y, h, rows.q.view(torch.uint8), rows.scale, g["dx"], g["dres"], g["dw"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(4):
        for name in ("x", "res", "dy", "dh"):
            d[name].normal_()
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
