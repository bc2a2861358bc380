"""Holder of one layer's experts as 8-bit floating-point codes (e4m3) with a
scale for each 128 x 128 block, and the layer's path over them.

Argument marshalling only: ``Fp8MoELayer.forward`` is the library's norm, route,
union and expert-FFN calls one after the other on one stream.  The holder's
methods make the arrays between those calls; they belong to the stream that the
calls run on, and so do the tensors that are returned.
"""
from __future__ import annotations

import torch

from ._lib import (_BF16, _E4M3, _F32, COLI_ERR_INVALID_ARG, COLI_ERR_UNSUPPORTED, ColiError, _stream_scope,
                   coli_add_rmsnorm_fp8, coli_moe_dims, coli_moe_expert_ffn_fp8, coli_moe_fp8_workspace_bytes,
                   coli_moe_route, coli_moe_union, coli_moe_weights_fp8)

_BLOCK = 128


def fp8_weights(gate_q, up_q, down_q, gate_s, up_s, down_s) -> coli_moe_weights_fp8:
    """The C struct of an expert set: codes e4m3 (or their bytes) gate/up [E+S, I,
    H] and down [E+S, H, I], scales fp32 [E+S, I/128, H/128] and [E+S, H/128,
    I/128], all on one device.  The tensors stay the caller's: keep them alive while
    it is used."""
    n, I, H = gate_q.shape
    nh, ni = H // _BLOCK, I // _BLOCK
    named = (("gate_q", gate_q, (n, I, H), _E4M3), ("up_q", up_q, (n, I, H), _E4M3), ("down_q", down_q, (n, H, I), _E4M3),
             ("gate_s", gate_s, (n, ni, nh), _F32), ("up_s", up_s, (n, ni, nh), _F32), ("down_s", down_s, (n, nh, ni), _F32))
    for name, t, shape, types in named:
        if t.shape != shape or t.dtype not in types:
            names = " or ".join(str(x).replace("torch.", "") for x in types)
            raise ValueError(f"{name}: {tuple(t.shape)} of {t.dtype}, needs {shape} of {names}")
    for name, t, *_ in named:
        if not t.is_contiguous() or not t.is_cuda:
            raise ValueError("the experts' codes and scales must be dense tensors in device memory")
        if t.get_device() != gate_q.get_device():
            raise ValueError(f"{name}: a tensor on {t.device}, but gate_q is on {gate_q.device}")
    w = coli_moe_weights_fp8(gate_q.data_ptr(), up_q.data_ptr(), down_q.data_ptr(), gate_s.data_ptr(),
                             up_s.data_ptr(), down_s.data_ptr())
    w.made_of = (n, I, H, gate_q.get_device())      # compared with the dims and the device of each call
    return w


class Fp8MoELayer:
    """One layer's e4m3 experts with the norm before them.

    dims: ``dims_for(H, I, E, k, S, group=128, code_bits=8)``; tensors: the six
    of ``fp8_weights`` by name; norm_weight: bf16 [H] or None."""

    def __init__(self, dims: coli_moe_dims, tensors: dict, norm_weight: torch.Tensor | None = None, eps: float = 1e-6):
        self.dims, self.t = dims, dict(tensors)
        n = dims.n_experts + dims.n_shared
        want = (n, dims.inter, dims.hidden)
        if tuple(self.t["gate_q"].shape) != want:
            raise ValueError(f"gate_q: {tuple(self.t['gate_q'].shape)}, the dims need {want}")
        self.weights = fp8_weights(**{m: self.t[m] for m in ("gate_q", "up_q", "down_q", "gate_s", "up_s", "down_s")})
        if norm_weight is not None:
            if norm_weight.numel() != dims.hidden or norm_weight.dtype not in _BF16:
                raise ValueError(f"norm_weight: {norm_weight.numel()} elements of {norm_weight.dtype}, the dims need "
                                 f"{dims.hidden} of bfloat16")
            if not norm_weight.is_contiguous() or norm_weight.get_device() != self.weights.made_of[3]:
                raise ValueError(f"norm_weight: needs a dense tensor on cuda:{self.weights.made_of[3]}")
        self.norm_weight, self.eps = norm_weight, eps

    def workspace(self, t_max: int, device="cuda") -> torch.Tensor:
        """Scratch for any call of up to ``t_max`` tokens."""
        n = coli_moe_fp8_workspace_bytes(self.dims, t_max)
        if n == 0:
            raise ColiError(COLI_ERR_INVALID_ARG if t_max < 0 else COLI_ERR_UNSUPPORTED, "coli_moe_fp8_workspace_bytes")
        return torch.empty(n, dtype=torch.uint8, device=device)

    def norm(self, x, residual=None, sum_out=None, norm_out=None, stream=None):
        """(codes, scales) of the normalised rows of x (+ residual)."""
        T, H = x.shape
        with _stream_scope(stream, x.device):
            q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=x.device)
            s = torch.empty((T, H // _BLOCK), dtype=torch.float32, device=x.device)
            coli_add_rmsnorm_fp8(x, residual, self.norm_weight, self.eps, sum_out, norm_out, q, s, stream)
        return q, s

    def experts(self, q, s, topk_ids, topk_w, out, ws, residual=None, stream=None):
        """Union, expert FFN and combine of a routed batch of codes ``q`` with scales ``s``."""
        T, E, P = q.shape[0], self.dims.n_experts, topk_ids.numel()
        new = lambda n: torch.empty(n, dtype=torch.int32, device=q.device)  # noqa: E731
        with _stream_scope(stream, q.device):
            unique, n_unique, seg, perm, pos = new(min(E, P)), new(1), new(min(E, P) + 1), new(P), new(P)
            if T:
                coli_moe_union(topk_ids, E, unique, n_unique, seg, perm, pos, stream)
                coli_moe_expert_ffn_fp8(self.dims, self.weights, q, s, topk_ids, topk_w, unique, n_unique, seg, perm,
                                        pos, residual, out, ws, stream)
        return out

    def forward(self, x, logits, out, ws, bias=None, residual=None, stream=None):
        """out = x' + experts(norm(x')), x' = x + residual, routed by ``logits``
        fp32 [T, E] (+ bias).  Returns (topk_ids, topk_w).

        A router that reads the normalised row goes call by call, with one norm:
        ``q, s = norm(x, residual, h, n)``, the logits from n, ``coli_moe_route``,
        ``experts(q, s, ids, w, out, ws, h)``."""
        T, k = x.shape[0], self.dims.top_k
        with _stream_scope(stream, x.device):
            h = x if residual is None else torch.empty_like(x)
            q, s = self.norm(x, residual, None if residual is None else h, None, stream)
            ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
            w = torch.empty((T, k), dtype=torch.float32, device=x.device)
            coli_moe_route(logits, bias, ids, w, stream)
            self.experts(q, s, ids, w, out, ws, h, stream)
        return ids, w
