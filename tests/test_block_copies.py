"""Copies of packed weights and of 8-bit rows: deep ones, pickled ones and
saved ones have memory of their own, which their calls read and write."""
import copy
import io
import pickle

import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.block import Linear4, Rows8

DEV = "cuda:0"


def saved(v):
    f = io.BytesIO()
    torch.save(v, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


COPIES = {"deepcopy": copy.deepcopy, "pickle": lambda v: pickle.loads(pickle.dumps(v)), "save": saved}


def proj(n=8, k=64, device="cpu", seed=0):
    p = Linear4.__new__(Linear4)
    p._make(n, k, torch.zeros(1, device=device))
    p.w4.packed.copy_(torch.randint(0, 120, p.w4.packed.shape, generator=torch.Generator().manual_seed(seed)))
    return p


def rows8(kind, T=3, n=64, device="cpu"):
    g = torch.Generator().manual_seed(1)
    q = torch.randn(T, n, generator=g).to(torch.float8_e4m3fn)
    s = torch.randint(120, 130, (T, n // 32), generator=g, dtype=torch.int64).to(torch.uint8)
    if kind == "given":
        return Rows8(q.to(device), s.to(device), torch.float32)
    if kind == "strided":
        wide, ws = torch.zeros(T, n + 32).to(torch.float8_e4m3fn).to(device), torch.zeros(T, 9, dtype=torch.uint8, device=device)
        wide[:, :n], ws[:, 1:1 + n // 32] = q.to(device), s.to(device)
        return Rows8(wide[:, :n], ws[:, 1:1 + n // 32], torch.float32)
    r = Rows8.empty(T, n, torch.float32, torch.zeros(1, device=device))
    r._memory[:T * n].copy_(q.view(torch.uint8).flatten())
    r._memory[T * n:].copy_(s.flatten())
    if kind == "seen":                     # its tensors were asked for before
        r.q, r.scale
    return r


def bytes_of(r):
    return r.q.view(torch.uint8).cpu().clone(), r.scale.cpu().clone()


@pytest.mark.parametrize("how", COPIES)
def test_copied_weights_name_their_own_memory(how):
    p = proj()
    before = p.w4.packed.clone()
    c = COPIES[how](p)
    assert (c.n, c.k, c.w4.n, c.w4.k) == (8, 64, 8, 64)
    assert c.w4.args == (c.w4.packed.data_ptr(), c.w4.packed.numel())
    assert c.w4.args[0] != p.w4.args[0] and torch.equal(c.w4.packed, before)
    c.w4.packed.zero_()
    assert torch.equal(p.w4.packed, before)


@pytest.mark.parametrize("how", COPIES)
@pytest.mark.parametrize("kind", ["given", "strided", "empty", "seen"])
def test_copied_rows_name_their_own_memory(kind, how):
    r = rows8(kind)
    q, s = bytes_of(r)
    c = COPIES[how](r)
    assert (c.shape, c.dtype, c.device) == (r.shape, r.dtype, r.device)
    assert c.ptrs[0] != r.ptrs[0] and c.ptrs[2] != r.ptrs[2]
    assert (c.ptrs[1], c.ptrs[3]) == (r.ptrs[1], r.ptrs[3])
    assert c.ptrs == (c.q.data_ptr(), c.ptrs[1], c.scale.data_ptr(), c.ptrs[3])
    assert torch.equal(c.q.view(torch.uint8), q) and torch.equal(c.scale, s)
    c.scale.zero_()
    assert torch.equal(r.scale, s)
    assert r.ptrs == (r.q.data_ptr(), r.ptrs[1], r.scale.data_ptr(), r.ptrs[3])


def test_weights_follow_their_tensor():
    """Packed weights that are put elsewhere, as a load or a move between
    devices puts them."""
    p = proj()
    p.w4.packed = p.w4.packed.clone()
    assert p.w4.args == (p.w4.packed.data_ptr(), p.w4.packed.numel())
    assert (p.w4.device, p.w4.index) == (p.w4.packed.device, -1)
    p.w4.packed = p.w4.packed.to("meta")
    assert p.w4.device.type == "meta"


def test_weights_that_are_not_in_a_row_are_refused():
    """Their size says nothing of the memory behind the address."""
    p = proj()
    p.w4.packed = p.w4.packed[:1].expand(p.w4.packed.numel())
    with pytest.raises(ValueError, match="contiguous"):
        p.w4.args


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES)
def test_copies_on_the_device(how):
    """A copy is packed anew and multiplies by its own weights; the original
    keeps its weights, and a copy outlives it."""
    g = torch.Generator().manual_seed(2)
    n, k = 40, 544
    W, V = ((torch.randn(n, k, generator=g) * s).to(torch.bfloat16).to(DEV) for s in (0.02, 0.5))
    x = torch.randn(5, k, generator=g).to(torch.bfloat16).to(DEV)
    p = Linear4(W)
    y, dense = p(x), p.weight()
    c = COPIES[how](p)
    assert torch.equal(c(x), y) and torch.equal(c.weight(), dense)
    L.gdn_w4_pack(V, c.w4)
    assert torch.equal(p(x), y) and torch.equal(p.weight(), dense)
    assert torch.equal(c.weight(), Linear4(V).weight())
    c = COPIES[how](p)
    del p
    torch.cuda.empty_cache()
    torch.empty(1 << 24, dtype=torch.uint8, device=DEV).fill_(255)
    assert torch.equal(c(x), y)


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES)
@pytest.mark.parametrize("kind", ["given", "strided", "empty", "seen"])
def test_copied_rows_on_the_device(kind, how):
    p = proj(40, 64, DEV)
    r = rows8(kind, device=DEV)
    y = p(r)
    c = COPIES[how](r)
    assert torch.equal(p(c), y)
    c.q.zero_()
    assert (p(c) == 0).all() and torch.equal(p(r), y)
