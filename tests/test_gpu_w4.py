"""4-bit weights: packing against the rule in 64 bits, products against sums
in 64 bits.

Products: codes, scales and the rows' values are taken exactly, so a sum of k
products carries the roundings of its additions only.  A matrix instruction
adds 32 products (128 for 8-bit rows) to a running sum; its additions round or
cut, 2^-23 of the partial sums at most, and those are bounded by S = sum |x w|.
With `terms` instructions in a row for each 32 inputs (one, two and three for
bf16, fp16 and fp32 rows) and the join of up to 32 partial sums this is
(terms (k / 32) + 32 + 32) 2^-23 S, or (k / 128 + 128 + 32) 2^-23 S, and half
a step of the output's type.

For 8-bit rows the instruction adds the products of eight adjacent inputs with
13 bits below the largest: with e(v) the exponent of a value (not below that of
the format's smallest normal one) each of the other seven is cut to a multiple
of 2^(max e(x) + e(w) - 13).  Seen on the device: beside 256 * 1 the product
2^-5 counts and 2^-6 does not, 256 * 6 + 2^-5 * 6 gives 1536.125, and inputs
eight apart add in full.  So 7 * 2^-13 of the largest 2^(e(x) + e(w)) of each
eight is added to what a sum may be off (`cut`).
"""
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import Linear4, Rows8

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TERMS = {"bf16": 1, "fp16": 2, "fp32": 3}
MAG = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
# rows, outputs, inputs: single ones, tails of every kind, the sizes of a layer's projections
SIZES = [(1, 1, 32), (1, 16, 512), (2, 17, 64), (3, 15, 480), (16, 50, 544), (17, 33, 1056), (1, 1544, 2560),
         (5, 1544, 2560), (9, 640, 6144), (33, 48, 1504), (40, 100, 8224), (64, 333, 2560), (130, 40, 96), (1, 8, 16416),
         (1, 8200, 512), (7, 8208, 1056), (30, 8216, 544), (70, 8200, 1568),
         (20, 8190, 4128), (33, 8100, 608), (100, 10250, 544), (300, 4100, 96),
         (14, 100, 2080), (4, 16400, 544), (8, 9000, 4128), (2, 100, 16928), (10, 50, 12320), (16, 40, 8192), (15, 33, 6656)]


def half(dt):
    return torch.finfo(dt).eps / 2


def make_codes(n, k, seed, lo=110, hi=130):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    scales = torch.randint(lo, hi, (n, k // 32), generator=g, dtype=torch.int64).to(torch.uint8)
    return codes, scales


def values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    v = MAG[c & 7] * (1 - 2 * (c >> 3))
    unit = torch.tensor(2.0, dtype=torch.float64) ** (scales.double() - 127)
    return v * unit.repeat_interleave(32, 1)


def rows_of(T, k, dt, seed, pad=0):
    g = torch.Generator().manual_seed(seed + 100)
    t = torch.full((T, k + pad), float("nan")).to(dt)
    t[:, :k] = torch.randn(T, k, generator=g).to(dt)
    return t.to(DEV)[:, :k]


def rows8_of(T, k, dt, seed, pad=0):
    g = torch.Generator().manual_seed(seed + 200)
    q = torch.full((T, k + pad), float("nan"))
    q[:, :k] = (torch.randn(T, k, generator=g) * 100).clamp(-448, 448)
    s = torch.full((T, k // 32 + pad), 255, dtype=torch.uint8)
    s[:, :k // 32] = torch.randint(115, 125, (T, k // 32), generator=g, dtype=torch.int64).to(torch.uint8)
    return Rows8(q.to(torch.float8_e4m3fn).to(DEV)[:, :k], s.to(DEV)[:, :k // 32], dt)


def values8(r):
    unit = torch.tensor(2.0, dtype=torch.float64) ** (r.scale.cpu().double() - 127)
    return r.q.cpu().double() * unit.repeat_interleave(32, 1)


def cut(r, codes, scales):
    """What the eights of 8-bit rows' products may lose, [T, n]."""

    def top(v, least, scale):          # 2^e(v) under the group's scale, 0 for 0
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** least)))
        return torch.where(v == 0, 0.0, torch.exp2(e)) * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)

    one = torch.full_like(scales, 127)
    x = top(r.q.double(), -6, r.scale)
    w = top(values(codes, one).to(DEV), 0, scales.to(DEV))
    lost = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=DEV)
    for a in range(0, x.shape[1], 8):
        lost += (x[:, None, a:a + 8] * w[None, :, a:a + 8]).amax(2)
    return (lost * 7 * 2.0 ** -13).cpu()


def check(y, xv, W, adds, more=0.0):
    ref, size = xv @ W.t(), xv.abs() @ W.abs().t()
    t = y.dtype
    tol = (half(t) * ref.abs() + adds * 2.0 ** -23 * size + more
           + torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
    got = y.cpu().double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all() and ((got - ref).abs() <= tol).all(), \
        f"off by {float(((got - ref).abs() / tol).max()):.3g} of what it may be"


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n,k", SIZES)
def test_product(T, n, k, dt):
    codes, scales = make_codes(n, k, T + n + k)
    x = rows_of(T, k, DT[dt], T)
    y = Linear4.from_codes(codes.to(DEV), scales.to(DEV))(x)
    assert y.dtype == DT[dt]
    check(y, x.cpu().double(), values(codes, scales), TERMS[dt] * (k // 32) + 64)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n,k", SIZES)
def test_product_of_8_bit_rows(T, n, k, dt):
    codes, scales = make_codes(n, k, T + n + k, 110, 125)
    r = rows8_of(T, k, DT[dt], T)
    y = Linear4.from_codes(codes.to(DEV), scales.to(DEV))(r)
    assert y.dtype == DT[dt]
    check(y, values8(r), values(codes, scales), k // 128 + 160, cut(r, codes, scales))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n,k", [(520, 4100, 544), (1030, 2057, 1056), (2050, 4100, 96)])
def test_prompts(T, n, k, dt):
    """Rows in hundreds and thousands, in 16 or 32 bits and in 8, into rows of
    a wider buffer: last rows, outputs and inputs end inside tiles."""
    codes, scales = make_codes(n, k, T + n + k, 110, 125)
    proj, W = Linear4.from_codes(codes.to(DEV), scales.to(DEV)), values(codes, scales)
    wide = n // 8 * 8 + 16
    for eight in (False, True):
        out = torch.full((T + 1, wide), 7.0, dtype=DT[dt], device=DEV)
        y = out[:T, :n]
        if eight:
            r = rows8_of(T, k, DT[dt], T, 48)
            L.w4_fwd_rows8(r, proj.w4, y)
            check(y, values8(r), W, k // 128 + 160, cut(r, codes, scales))
        else:
            x = rows_of(T, k, DT[dt], T, 24)
            L.gdn_w4_fwd(x, proj.w4, y)
            check(y, x.cpu().double(), W, TERMS[dt] * (k // 32) + 64)
        assert (out[T:] == 7).all() and (out[:, n:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_every_code_value_and_position(dt):
    """Rows with a single one pick the weights out one by one, exactly."""
    n, k = 16, 544
    codes, scales = make_codes(n, k, 5, 118, 134)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    W = values(codes, scales)
    assert torch.equal(proj.weight(DT[dt]).cpu().double(), W)
    assert torch.equal(proj(torch.eye(k, dtype=DT[dt], device=DEV)).cpu().double(), W.t())
    one = torch.eye(k).to(torch.float8_e4m3fn).to(DEV)
    unit = torch.full((k, k // 32), 127, dtype=torch.uint8, device=DEV)
    assert torch.equal(proj(Rows8(one, unit, DT[dt])).cpu().double(), W.t())


@pytest.mark.parametrize("T", [1, 5, 33])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rows_of_wider_buffers(T, dt):
    """Strided rows; between them nothing is read (NaN) or written."""
    n, k = 43, 544
    codes, scales = make_codes(n, k, 6)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    for x, v, adds in ((rows_of(T, k, DT[dt], 1, 40), None, 3 * (k // 32) + 64),
                       (rows8_of(T, k, DT[dt], 1, 16), 8, k // 128 + 160)):
        y0 = torch.full((T + 2, 64), 7.0, dtype=DT[dt], device=DEV)
        y = y0[1:-1, 8:8 + n]
        if v is None:
            L.gdn_w4_fwd(x, proj.w4, y)
            v = x.cpu().double()
        else:
            L.gdn_w4_fwd_mx8(x.q, x.scale, proj.w4, y)
            v = values8(x)
        check(y, v, values(codes, scales), adds, cut(x, codes, scales) if isinstance(x, Rows8) else 0.0)
        assert (y0[0] == 7).all() and (y0[-1] == 7).all() and (y0[:, :8] == 7).all() and (y0[:, 8 + n:] == 7).all()


def test_strided_codes_and_scales():
    n, k = 21, 96
    codes, scales = make_codes(n, k, 7)
    c0 = torch.zeros(n, 64, dtype=torch.uint8)
    s0 = torch.full((n, 5), 255, dtype=torch.uint8)
    c0[:, :k // 2], s0[:, 1:1 + k // 32] = codes, scales
    proj = Linear4.from_codes(c0.to(DEV)[:, :k // 2], s0.to(DEV)[:, 1:1 + k // 32])
    assert torch.equal(proj.weight(torch.float32).cpu().double(), values(codes, scales))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_not_finite_rows_stay_alone(dt):
    n, k = 40, 640
    codes, scales = make_codes(n, k, 8)
    codes |= 0x11                                     # no weight is zero: inf * w = inf
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    x = rows_of(20, k, DT[dt], 2)
    x[3, 100], x[17, 639] = float("nan"), float("inf")
    y = proj(x)
    assert y[3].isnan().all() and torch.isinf(y[17]).all()
    W = values(codes, scales)
    assert torch.equal(torch.signbit(y[17].cpu()), W[:, 639] < 0)
    keep = [i for i in range(20) if i not in (3, 17)]
    check(y[keep], x[keep].cpu().double(), W, TERMS[dt] * (k // 32) + 64)
    r = rows8_of(20, k, DT[dt], 3)
    q = r.q.view(torch.uint8)
    q[3, 100] = 0x7f                                  # NaN
    r.scale[17, 4] = 255                              # a group of NaN
    y = proj(r)
    assert y[3].isnan().all() and y[17].isnan().all()
    r.scale[17, 4], q[3, 100] = 120, 0
    check(y[keep], values8(r)[keep], W, k // 128 + 160, cut(r, codes, scales)[keep])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_scales_at_the_ends(dt):
    """Bytes 1 and 253 with rows that bring the products back; 255 is NaN."""
    n, k = 16, 64
    codes, _ = make_codes(n, k, 9)
    codes |= 0x11
    scales = torch.full((n, 2), 127, dtype=torch.uint8)
    x = rows_of(3, k, torch.float32, 4)
    for byte, up in ((3, 2.0 ** 100), (250, 2.0 ** -100)):
        scales[:, 0] = byte
        scales[:, 1] = byte
        xs = (x * up).to(DT[dt])
        proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
        check(proj(xs), xs.cpu().double(), values(codes, scales), 3 * 2 + 64)
    scales[:] = 127
    scales[5, 1] = 255
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    y = proj(x.to(DT[dt]))
    assert y[:, 5].isnan().all() and y[:, :5].isfinite().all() and y[:, 6:].isfinite().all()
    w = proj.weight(DT[dt])
    assert w[5, 32:].isnan().all() and w[5, :32].isfinite().all()


@pytest.mark.parametrize("T", [1, 7, 40])
def test_fp16_rows_by_weights_that_fp16_does_not_hold(T):
    """Scales just inside and just outside of what fp16 holds exactly, and far
    outside, next to each other; rows bring the products back into range."""
    n, k = 64, 1056
    codes, _ = make_codes(n, k, 16)
    g = torch.Generator().manual_seed(17)
    for lo, hi in ((113, 117), (138, 142), (114, 115), (140, 141), (20, 60), (0, 1)):
        scales = torch.full((n, k // 32), 127, dtype=torch.uint8)
        scales[:, 5::7] = torch.randint(lo, hi, scales[:, 5::7].shape, generator=g, dtype=torch.int64).to(torch.uint8)
        proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
        x = rows_of(T, k, torch.float16, 18) * (2.0 ** -12 if lo > 127 else 1.0)
        check(proj(x), x.cpu().double(), values(codes, scales), 2 * (k // 32) + 64)
        only = torch.zeros(n, k // 32, dtype=torch.bool)
        only[:, 5::7] = True
        c2 = torch.where(only.repeat_interleave(16, 1), codes, 0)
        y = Linear4.from_codes(c2.to(DEV), scales.to(DEV))(x)
        check(y, x.cpu().double(), values(c2, scales), 2 * (k // 32) + 64)


def test_values_across_the_types_ranges():
    """fp16 and fp32 rows enter whole: the smallest and largest of their
    values, next to each other."""
    n, k = 16, 64
    codes, scales = make_codes(n, k, 10, 120, 128)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    W = values(codes, scales)
    for dt, v in (("fp16", [65504, 6.1e-5, 5.96e-8, -65504, 1.0009765625, 0]),
                  ("fp32", [1e30, 1 + 2.0 ** -23, 1e-30, -1e30, 3.1415927, 0])):
        for one in v:
            x = torch.zeros(1, k, dtype=DT[dt], device=DEV)
            x[0, 37] = one
            y = proj(x.to(DT[dt])) if dt == "fp32" else None
            out = torch.empty(1, n, dtype=DT[dt], device=DEV) if y is None else y
            if y is None:
                L.gdn_w4_fwd(x, proj.w4, out)
            check(out if dt == "fp32" else out.clamp(-65504, 65504), x.cpu().double(),
                  W if dt == "fp32" else W.clamp(-65504 / max(abs(one), 1), 65504 / max(abs(one), 1)), 3 * 2 + 64)


def test_no_rows():
    codes, scales = make_codes(24, 64, 11)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    assert proj(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)).shape == (0, 24)
    r = Rows8(torch.empty(0, 64, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(0, 2, dtype=torch.uint8, device=DEV))
    assert proj(r).shape == (0, 24)


@pytest.mark.parametrize("k", [64, 2560, 8224])
def test_repeats_bit_by_bit(k):
    n = 200
    codes, scales = make_codes(n, k, 12)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    for x in (rows_of(30, k, torch.bfloat16, 5), rows8_of(30, k, torch.bfloat16, 5)):
        y = proj(x)
        assert all(torch.equal(proj(x), y) for _ in range(4))


def test_weights_beyond_32_bits():
    """More than 2^32 bytes of codes: outputs here and there."""
    n, k = (1 << 22) - 5, 2080
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV).random_(0, 256, generator=g)
    scales = torch.empty(n, k // 32, dtype=torch.uint8, device=DEV).random_(118, 122, generator=g)
    proj = Linear4.from_codes(codes, scales)
    at = [0, 15, 16, 1000, (1 << 21) + 7, (1 << 22) - 20, n - 17, n - 1]
    W = values(codes[at].cpu(), scales[at].cpu())
    for T in (1, 3, 20):
        x = rows_of(T, k, torch.bfloat16, T)
        check(proj(x)[:, at].contiguous(), x.cpu().double(), W, k // 32 + 64)
    r = rows8_of(2, k, torch.bfloat16, 5)
    check(proj(r)[:, at].contiguous(), values8(r), W, k // 128 + 160, cut(r, codes[at].cpu(), scales[at].cpu()))


# ------------------------------------------------------------------ packing
def ref_pack(W):
    """The values that W's 4-bit form stands for, and the scales' bytes."""
    g = W.double().reshape(W.shape[0], -1, 32)
    amax = g.abs().amax(2, keepdim=True)
    m, e = torch.frexp(amax)
    # at most 2^125: 4 * 2^126 = 2^128 is beyond fp32, 6 * 2^125 < 2^128 - 2^104 is not
    e = (e - 3 + (m > 0.75)).clamp(-127, 125).masked_fill(amax == 0, -127)

    def at(e):
        unit = torch.tensor(2.0, dtype=torch.float64) ** e.double()
        a = (g / unit).abs()
        c = torch.zeros_like(a, dtype=torch.long)
        for i in range(7):
            mid = (MAG[i] + MAG[i + 1]) / 2
            c = torch.where((a >= mid) if i % 2 else (a > mid), i + 1, c)
        v = MAG[c] * torch.sign(g) * unit
        return v, (v - g).square().sum(2, keepdim=True)

    (v1, s1), (v2, s2) = at(e), at((e - 1).clamp(min=-127))
    less = s2 < s1
    return torch.where(less, v2, v1).reshape(W.shape), torch.where(less, e - 1, e)[:, :, 0] + 127


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,k,pad", [(1, 32, 0), (16, 512, 0), (17, 544, 8), (50, 96, 40), (333, 2560, 0)])
def test_pack(n, k, pad, dt):
    W = rows_of(n, k, DT[dt], n, pad)
    W *= 0.02
    proj = Linear4(W)
    want, _ = ref_pack(W.cpu())
    assert torch.equal(proj.weight(torch.float32).cpu().double(), want)
    assert torch.equal(proj.weight(DT[dt]).cpu().double(), want)


def test_pack_ties_and_edges():
    """Every tie of the format, cut values, groups of zeros, of one value,
    of the smallest and largest numbers; NaN and infinities."""
    W = torch.zeros(12, 64)
    W[0, :9] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25])
    W[1, :9] = -W[0, :9]
    W[2, :32] = 7.0                                      # 6 is nearer than 8 under the larger scale
    W[3, :32] = torch.tensor([7.0] + [0.5] * 31)         # cutting 7 to 6 keeps the small ones
    W[4, 32:] = 1e-30
    W[5, 32:] = 3e38
    W[6, 5] = 2.0 ** -126
    W[7, 40:50] = torch.linspace(-1, 1, 10)
    W[8] = torch.randn(64, generator=torch.Generator().manual_seed(1)) * 1e-38
    proj = Linear4(W.to(DEV))
    want, bytes_ = ref_pack(W[:10])
    got = proj.weight(torch.float32).cpu().double()
    assert torch.equal(got[:10], want)
    assert torch.equal(got[0, :9], torch.tensor([6, 0, 1, 1, 2, 2, 4, 4, 0], dtype=torch.float64))
    W[10, 3], W[11, 35] = float("nan"), -float("inf")
    got = Linear4(W.to(DEV)).weight(torch.float32).cpu().double()
    assert got[10, :32].isnan().all() and got[11, 32:].isnan().all()
    assert (got[10, 32:] == 0).all() and (got[11, :32] == 0).all() and torch.equal(got[:10], want)


def test_pack_then_product():
    W = rows_of(100, 1056, torch.bfloat16, 13) * 0.05
    x = rows_of(7, 1056, torch.bfloat16, 14)
    proj = Linear4(W)
    check(proj(x), x.cpu().double(), ref_pack(W.cpu())[0], 1056 // 32 + 64)


# ------------------------------------------------------------------ streams and graphs
def test_other_streams_and_replays():
    n, k, T = 1544, 2560, 20
    codes, scales = make_codes(n, k, 15)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    x, r = rows_of(T, k, torch.bfloat16, 6), rows8_of(T, k, torch.bfloat16, 6)
    want = proj(x), proj(r)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for s, v in zip(streams, (x, r)):
            with torch.cuda.stream(s):
                got.append(proj(v))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = proj(x), proj(r)
    for i in range(4):
        x.normal_()
        r.scale.random_(110, 125)
        want = proj(x), proj(r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i
