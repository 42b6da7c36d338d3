"""What stands around the core in a model's block, on top of libgdn: the
residual's addition with the zero-centred RMSNorm before a layer (forward,
forward into 8 bits, backward), projections with weights of 4 bits, and the
served layer made of them.

As in layer.py this only allocates with torch and calls the C ABI.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import capi as L
from .capi import Rows8
from .layer import GDNCore

__all__ = ["ResidualNorm", "Rows8", "Linear4", "GDNLayer4"]


class ResidualNorm:
    """h = x + res, y = h / sqrt(mean h^2 + eps) * (1 + w) over rows of
    `hidden` columns.  x and y are of `dtype`, the residual stream (res, h) of
    res_dtype: the same (the default) or fp32.  Rows may be strided.  Every
    call has outputs and scratch of its own, and nothing synchronises."""

    def __init__(self, hidden: int, dtype: torch.dtype = torch.bfloat16,
                 res_dtype: Optional[torch.dtype] = None, eps: float = 1e-6, device="cuda"):
        if hidden < 8 or hidden % 8:
            raise ValueError(f"rows of {hidden} columns: a multiple of 8 is needed")
        self.hidden, self.dtype, self.eps = hidden, dtype, eps
        self.res_dtype = dtype if res_dtype is None else res_dtype
        L._types(self.dtype, self.res_dtype)
        self.device = torch.device(device)
        L.load()

    def _sum(self, x, res):
        """Where h goes: new memory; x itself where nothing is added or converted."""
        if x.dtype is not self.dtype or x.dim() != 2 or x.shape[1] != self.hidden:
            raise ValueError(f"x must be {self.dtype} [T, {self.hidden}], got {x.dtype} {tuple(x.shape)}")
        if res is not None and res.dtype is not self.res_dtype:
            raise TypeError(f"res must be {self.res_dtype}, got {res.dtype}")
        if res is None and self.dtype is self.res_dtype:
            return None
        return torch.empty_like(x if res is None else res, dtype=self.res_dtype)

    def forward(self, x, res, w):
        """-> (y, h).  res None: h is x, in the stream's type."""
        h = self._sum(x, res)
        y = torch.empty_like(x)
        L.gdn_add_norm_fwd(x, res, w, h, y, self.eps)
        return y, x if h is None else h

    def forward8(self, x, res, w):
        """-> (Rows8, h): y in 8 bits, for Linear4.  hidden a multiple of 32."""
        h = self._sum(x, res)
        rows = Rows8.empty(x.shape[0], self.hidden, self.dtype, x)
        L.add_norm_fwd_rows8(x, res, w, h, rows, self.eps)
        return rows, x if h is None else h

    def backward(self, h, w, dy, dh=None):
        """From the forward's h: dy is y's gradient, dh that of h from where the
        stream goes on -> dict of dx (in dtype), dres (in res_dtype; the same
        tensor where the types are) and dw (fp32)."""
        if dy.dtype != self.dtype or h.dtype != self.res_dtype:
            raise TypeError(f"dy must be {self.dtype} and h {self.res_dtype}, got {dy.dtype} and {h.dtype}")
        dres = torch.empty_like(h)
        dx = torch.empty_like(dy) if self.dtype != self.res_dtype else None
        dw = h.new_empty(h.shape[-1], dtype=torch.float32)
        ws = h.new_empty(L.gdn_add_norm_bwd_workspace(h.shape[0], h.shape[-1]), dtype=torch.uint8)
        L.gdn_add_norm_bwd(h, w, dy, dh, dx, dres, dw, ws, self.eps)
        return {"dx": dres if dx is None else dx, "dres": dres, "dw": dw}


class Linear4:
    """A projection with weights of 4 bits (e2m1 under a power of two for each
    32 inputs), for few rows: Linear4(weight [N, K])(x [T, K]) -> [T, N]."""

    def __init__(self, weight: torch.Tensor):
        self._make(weight.shape[0], weight.shape[1], weight)
        L.gdn_w4_pack(weight, self.w4)

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor) -> "Linear4":
        """Weights that are in 4 bits already: codes uint8 [N, K / 2] (input 2j
        in the low four bits of byte j), scales uint8 [N, K / 32] (2^(byte - 127))."""
        self = cls.__new__(cls)
        self._make(codes.shape[0], 2 * codes.shape[1], codes)
        L.gdn_w4_arrange(codes, scales, self.w4)
        return self

    def _make(self, n, k, like):
        self.n, self.k = n, k
        self.w4 = L.W4(like, n, k, make=True)

    def weight(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The values [N, K] that the weights stand for, for a dense product
        of many rows."""
        w = self.w4.packed.new_empty((self.n, self.k), dtype=dtype)
        L.gdn_w4_unpack(self.w4, w)
        return w

    def __call__(self, x) -> torch.Tensor:
        """x: a tensor [T, K] of a storage type (rows may be strided) or Rows8.
        Where N is not a multiple of 8 the rows of the result are strided.  A
        row's last bits may depend on T, which the order of its sums follows."""
        rows, n = x.shape[0], self.n
        t = self.w4.packed if isinstance(x, Rows8) else x
        if n % 8 == 0:
            y = t.new_empty((rows, n), dtype=x.dtype)
        else:                           # the row stride is a multiple of 8
            y = t.new_empty_strided((rows, n), (n // 8 * 8 + 8, 1), dtype=x.dtype)
        if t is x:
            L.gdn_w4_fwd(x, self.w4, y)
        else:
            L.w4_fwd_rows8(x, self.w4, y)
        return y


class GDNLayer4:
    """GDNLayer's serving form with projections of 4 bits: hidden states X
    [T, H] (a tensor or Rows8, from ResidualNorm.forward8) -> Y [T, H].  The
    four input projections are one product, whose columns the core's step reads
    where they are: a layer's step is the norm, two products and the core's step.
    prefill copies the columns of z, a and b, which the chunked forward wants
    contiguous."""

    def __init__(self, cfg, hidden: int, weights: dict, device="cuda"):
        """weights: GDNLayer's, name -> [out, in] tensors."""
        self.core = GDNCore(cfg, device)
        self.cfg, self.hidden = cfg, hidden
        self.proj_in = Linear4(torch.cat([weights[k] for k in ("x", "z", "a", "b")], 0))
        self.proj_out = Linear4(weights["out"].contiguous())

    def split(self, P):
        """The input projections' columns: x, z, a, b."""
        c = self.cfg
        at = [0, c.channels, c.channels + c.hv * c.d, c.channels + c.hv * c.d + c.hv]
        return [P[:, s:e] for s, e in zip(at, at[1:] + [at[3] + c.hv])]

    def step(self, X, w_conv, A_log, dt_bias, w_norm, cu_seqlens, cache, slot_in, slot_out=None,
             slot_tok=None, layer=0):
        """The layer for the next tokens of cached sequences, as GDNLayer.step."""
        x, z, a, b = self.split(self.proj_in(X))
        out = self.core.step(x, w_conv, a, b, A_log, dt_bias, z, w_norm, cu_seqlens, cache, slot_in,
                             slot_out, slot_tok, layer)
        return self.proj_out(out.view(X.shape[0], self.cfg.hv * self.cfg.d))

    def prefill(self, X, w_conv, A_log, dt_bias, w_norm, cu_seqlens, cache, slot_in, slot_out=None,
                layer=0):
        """step() for prompts, through GDNCore.prefill (and copies of z, a and b)."""
        x, z, a, b = self.split(self.proj_in(X))
        out = self.core.prefill(x, w_conv, a.contiguous(), b.contiguous(), A_log, dt_bias,
                                z.contiguous(), w_norm, cu_seqlens, cache, slot_in, slot_out, layer)
        return self.proj_out(out.view(X.shape[0], self.cfg.hv * self.cfg.d))
