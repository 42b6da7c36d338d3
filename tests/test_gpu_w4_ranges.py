"""4-bit weights at the ends of their scales, and rows at the low end of
their types.  Tolerances as in test_gpu_w4; of fp32 rows what lies below
2^-133, bf16's smallest value, is cut, so a sum may lose 2^-133 sum |w| more."""
import pytest
import torch

from gated_deltanet_layer_causal_amd.block import Linear4, Rows8
from tests.test_gpu_w4 import DEV, DT, TERMS, check, cut, make_codes, values, values8

pytestmark = pytest.mark.gpu

N, K = 16, 64
BEYOND = {253: 4.0, 254: 2.0}          # the least magnitude that is 2^128 or more


def rows(T, up, dt, seed=4):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, K, generator=g).double() * up).to(DT[dt]).to(DEV)


def rows8(T, byte, dt, seed=4):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    return Rows8(q.to(DEV), torch.full((T, K // 32), byte, dtype=torch.uint8, device=DEV), DT[dt])


def weights(byte, most=6.0, seed=9):
    """Codes of magnitudes up to `most` under one byte: codes, scales, values."""
    codes, _ = make_codes(N, K, seed)
    codes |= 0x11                      # no zeros
    scales = torch.full((N, K // 32), byte, dtype=torch.uint8)
    one = values(codes, torch.full_like(scales, 127))
    small = torch.where(one.abs() <= most, codes_of(one), 1)
    codes = (small[:, 0::2] | small[:, 1::2] << 4).to(torch.uint8)
    return codes, scales, values(codes, scales)


def codes_of(v):
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    return torch.searchsorted(mag, v.abs()) + 8 * (v < 0)


def proj(codes, scales):
    return Linear4.from_codes(codes.to(DEV), scales.to(DEV))


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("byte", [0, 1, 2, 252])
def test_first_and_last_scales(byte, dt, T):
    """Weights from 2^-128 (no normal number) to 6 * 2^125, with rows that
    bring the products back."""
    codes, scales, W = weights(byte)
    p = proj(codes, scales)
    assert torch.equal(p.weight(DT[dt]).cpu().double(), W)
    x = rows(T, 2.0 ** (100 if byte < 127 else -100), dt)
    check(p(x), x.cpu().double(), W, TERMS[dt] * (K // 32) + 64)
    r = rows8(T, 227 if byte < 127 else 27, dt)
    check(p(r), values8(r), W, K // 128 + 160, cut(r, codes, scales))


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("byte", [253, 254])
def test_scales_whose_larger_values_are_beyond_fp32(byte, dt, T):
    """What fp32 holds is exact; what it does not is an infinity in dense
    weights, leaves no finite sum with 16- or 32-bit rows (fp32 rows enter in
    terms, of which one may be zero), and is itself with 8-bit rows."""
    fits = 3.0 if byte == 253 else 1.5
    codes, scales, W = weights(byte, fits)
    p = proj(codes, scales)
    assert torch.equal(p.weight(DT[dt]).cpu().double(), W)
    x = rows(T, 2.0 ** -100, dt)
    check(p(x), x.cpu().double(), W, TERMS[dt] * (K // 32) + 64)
    r = rows8(T, 27, dt)
    check(p(r), values8(r), W, K // 128 + 160, cut(r, codes, scales))

    codes, scales, W = weights(byte)
    out = W.abs() >= 2.0 ** 128
    assert out.any() and (out == (W.abs() >= BEYOND[byte] * 2.0 ** (byte - 127))).all()
    want = torch.where(out, torch.sign(W) * float("inf"), W)
    p = proj(codes, scales)
    assert torch.equal(p.weight(DT[dt]).cpu().double(), want)
    check(p(r), values8(r), W, K // 128 + 160, cut(r, codes, scales))
    assert not p(x)[:, out.any(1).to(DEV)].isfinite().any()


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("e", [-109, -112, -126, -130, -134])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rows_at_the_low_end(dt, e, T):
    """bf16 rows enter as they are, numbers below the normal ones too; of fp32
    rows what lies below 2^-133 is cut."""
    codes, scales, W = weights(227)
    x = rows(T, 2.0 ** e, dt)
    lost = 2.0 ** -133 * W.abs().sum(1) if dt == "fp32" else 0.0
    check(proj(codes, scales)(x), x.cpu().double(), W, TERMS[dt] * (K // 32) + 64, lost)


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("byte", [120, 135, 141])
def test_fp16_rows_below_the_normal_numbers(byte, T):
    codes, scales, W = weights(byte)
    x = rows(T, 2.0 ** -18, "fp16")
    assert (x.abs() < 2.0 ** -14).all() and (x != 0).any()
    check(proj(codes, scales)(x), x.cpu().double(), W, TERMS["fp16"] * (K // 32) + 64)
