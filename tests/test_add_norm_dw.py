"""dw of the residual norm's backward over many rows, with checks that a lost
workgroup cannot pass.

A column's terms dy n are added in a thread (its share of the rows), over the rows
side by side in a workgroup, then over the workgroups' partial sums, sixteen
chains and their join.  A sum that goes through `depth` additions is off by
depth 2^-24 sum |dy n| at most, and a term by 48 2^-24 of itself (its n: see
test_gpu_add_norm).  The longest chain is a few hundred additions however many
rows there are.

Rows of +-1 (eps 0, a power of two of columns) have rho = 1 exactly, so with
whole numbers as dy every sum below 2^24 is exact, in any order."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import ResidualNorm

DEV = "cuda:0"
U = 2.0 ** -24
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# rows, columns, types; the first five are beyond the cache, where rows are taken two at a time
RANDOM = [(349601, 72, "fp32", "fp32"), (95407, 264, "fp32", "fp32"), (70001, 480, "bf16", "fp32"),
          (105003, 512, "fp16", "fp16"), (211003, 256, "bf16", "bf16"), (20000, 256, "bf16", "bf16"),
          (30011, 40, "fp16", "fp32"), (9000, 2560, "bf16", "fp32"), (5000, 3200, "fp16", "fp16"),
          (2309, 4128, "bf16", "bf16"), (1031, 8192, "bf16", "fp32"), (777, 8200, "fp32", "fp32"),
          (1285, 16384, "fp16", "fp16")]


def blocks(T, n):
    """Workgroups that leave a partial sum."""
    return L.gdn_add_norm_bwd_workspace(T, n) // (4 * n)


def depth(T, n):
    side = 32 if n <= 64 else 8 if n <= 256 else 4 if n <= 512 else 1      # rows side by side
    g = blocks(T, n)
    return -(-T // (g * side)) + 2 + side + -(-g // 16) + 16


def bound(T, n, size):
    return (depth(T, n) + 48) * U * size


@pytest.mark.parametrize("T,n,dt,rt", RANDOM)
def test_the_bound_rejects_a_lost_workgroup(T, n, dt, rt):
    """On the host: what one workgroup adds (T / blocks rows) is beyond what the
    sums may be off in most columns; T additions' worth of roundings would
    let it pass in the longest shapes."""
    g = np.random.default_rng(n)
    t = g.standard_normal((T, 32)) * 2 * g.standard_normal((T, 32))
    share = t[: T // blocks(T, n)].sum(0)
    size = np.abs(t).sum(0)
    tol = bound(T, n, size)
    assert (np.abs(share) > 2 * tol).mean() > 0.7
    assert (tol < np.abs(t.sum(0)).mean() / 20).all()
    if T > 200000:
        assert (np.abs(share) < (T + 48) * U * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,dt,rt", RANDOM)
def test_dw_of_many_rows(T, n, dt, rt):
    g = torch.Generator(device=DEV).manual_seed(n)
    h = (torch.randn(T, n, generator=g, device=DEV) * 3).to(DT[rt])
    dy = (torch.randn(T, n, generator=g, device=DEV) * 2).to(DT[dt])
    w = torch.randn(n, generator=g, device=DEV) * 0.1
    eps = 1e-5
    dw = ResidualNorm(n, DT[dt], DT[rt], eps).backward(h, w, dy)["dw"].double()
    hd = h.double()
    t = dy.double() * hd * (hd.square().mean(1, keepdim=True) + eps).rsqrt()
    off, tol = (dw - t.sum(0)).abs(), bound(T, n, t.abs().sum(0))
    assert (off <= tol).all(), float((off / tol).max())


EXACT = [(30011, 64), (262147, 128), (20011, 128), (211003, 256), (105003, 512), (20011, 512), (3001, 1024), (3001, 2048),
         (3001, 4096), (1031, 8192), (777, 16384), (3, 64), (2, 1024), (513, 2048), (257, 8192), (255, 16384)]


def whole(T, n, dt, rt, most, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + n)
    h = torch.empty(T, n, dtype=DT[rt], device=DEV).random_(0, 2, generator=g).mul_(2).sub_(1)
    dy = torch.empty(T, n, dtype=DT[dt], device=DEV).random_(-most, most + 1, generator=g)
    return h, dy


@pytest.mark.gpu
@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("T,n", EXACT)
def test_whole_numbers_are_summed_exactly(T, n, dt, rt):
    h, dy = whole(T, n, dt, rt, 3)
    dw = ResidualNorm(n, DT[dt], DT[rt], 0.0).backward(h, torch.zeros(n, device=DEV), dy)["dw"]
    want = (dy.double() * h.double()).sum(0)
    assert want.abs().max() < 2 ** 24 and torch.equal(dw.double(), want)


@pytest.mark.gpu
def test_whole_numbers_of_more_than_2_32_values():
    T, n = (1 << 22) + 3, 1024
    h, dy = whole(T, n, "bf16", "bf16", 2)
    norm = ResidualNorm(n, eps=0.0)
    dw = torch.empty(n, device=DEV)
    ws = torch.empty(L.gdn_add_norm_bwd_workspace(T, n), dtype=torch.uint8, device=DEV)
    L.gdn_add_norm_bwd(h, torch.zeros(n, device=DEV), dy, None, None, None, dw, ws, norm.eps)
    want = torch.zeros(n, dtype=torch.float64, device=DEV)
    for a in range(0, T, 1 << 18):
        want += (dy[a:a + (1 << 18)].double() * h[a:a + (1 << 18)].double()).sum(0)
    assert torch.equal(dw.double(), want)
