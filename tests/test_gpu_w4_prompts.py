"""4-bit projections of prompts, with inputs enough that the two buffers of
staged rows and the weights asked for ahead change places several times: every
output against sums in 64 bits.  Tolerances as in test_gpu_w4."""
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import Linear4
from tests.test_gpu_w4 import DEV, DT, TERMS, cut, half, make_codes, rows8_of, rows_of, values, values8

pytestmark = pytest.mark.gpu

# rows, outputs, inputs: more than 32768 and 8192 tiles of 16 x 16, last steps half full and full
SIZES = [(2050, 4100, 1056), (4101, 2075, 2592), (1030, 2057, 4128)]


def check(y, x, W, adds, more=0.0):
    x, W = x.to(DEV), W.to(DEV)
    ref, size = x @ W.t(), x.abs() @ W.abs().t()
    t = y.dtype
    tol = half(t) * ref.abs() + adds * 2.0 ** -23 * size + more + torch.finfo(t).smallest_normal * half(t)
    off = (y.double() - ref).abs()
    assert torch.isfinite(y).all() and (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("lo,hi", [(118, 130), (105, 130)])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n,k", SIZES)
def test_rows_of_16_and_32_bits(T, n, k, dt, lo, hi):
    """Scales that fp16 holds the weights under, and others among them."""
    codes, scales = make_codes(n, k, T + n, lo, hi)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    x = rows_of(T, k, DT[dt], T, 24)
    out = torch.full((T + 2, n // 8 * 8 + 16), 7.0, dtype=DT[dt], device=DEV)
    L.gdn_w4_fwd(x, proj.w4, out[1:-1, :n])
    check(out[1:-1, :n], x.double(), values(codes, scales), TERMS[dt] * (k // 32) + 64)
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, n:] == 7).all()
    assert all(torch.equal(proj(x), out[1:-1, :n]) for _ in range(3))


@pytest.mark.parametrize("T,n,k", SIZES)
def test_rows_of_8_bits(T, n, k):
    codes, scales = make_codes(n, k, T + n, 110, 125)
    proj = Linear4.from_codes(codes.to(DEV), scales.to(DEV))
    r = rows8_of(T, k, torch.float32, T, 48)
    out = torch.full((T + 2, n // 8 * 8 + 16), 7.0, device=DEV)
    L.w4_fwd_rows8(r, proj.w4, out[1:-1, :n])
    check(out[1:-1, :n], values8(r), values(codes, scales), k // 128 + 160, cut(r, codes, scales).to(DEV))
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, n:] == 7).all()
    assert all(torch.equal(proj(r), out[1:-1, :n]) for _ in range(3))
