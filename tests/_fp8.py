"""Plain 64-bit statements of the 8-bit floating-point operators and the balance
loss for their tests.  Written from the formulas in include/coli_moe.h; they
share no code with the library."""
from __future__ import annotations

import numpy as np
import torch

F8 = torch.float8_e4m3fn
BLOCK = 128
U32 = 2.0 ** -24       # half a step of fp32
UBF16 = 2.0 ** -8      # half a step of bf16 (the value below a power of two: 2^-9 of it, 2^-8 at most)


def e4m3_values() -> np.ndarray:
    """The 256 values of the codes, from their bit fields (sign, 4 exponent bits
    with bias 7, 3 fraction bits; S.1111.111 is NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = float("nan") if (e == 15 and f == 7) else (-v if s else v)
    return out


VALUES = e4m3_values()


def decode(codes) -> torch.Tensor:
    """fp64 values of an e4m3 tensor (or its bytes)."""
    b = codes.contiguous().view(torch.uint8).cpu()
    return torch.from_numpy(VALUES)[b.long()]


def e4m3_round(v: torch.Tensor) -> torch.Tensor:
    """fp64 -> nearest e4m3 value (ties to the even code), saturating."""
    grid = torch.from_numpy(VALUES[:127])                 # 0 .. 448 ascending
    a = v.abs().clamp_max(448.0)
    hi = torch.searchsorted(grid, a).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], v)


def spread(s: torch.Tensor, n: int, dim: int) -> torch.Tensor:
    return torch.repeat_interleave(s, BLOCK, dim=dim).narrow(dim, 0, n)


def a_values(q, s):
    return decode(q) * spread(s.double().cpu(), q.shape[-1], -1)


def w_values(q, s):
    full = spread(spread(s.double().cpu(), q.shape[-2], -2), q.shape[-1], -1)
    return decode(q) * full


def block_quantise(v: torch.Tensor, rows: int):
    """Codes and scales of fp64 values [..., R, K], a scale for each rows x 128
    block (the test inputs' maker: any codes and scales would do)."""
    R, K = v.shape[-2:]
    p = torch.nn.functional.pad(v, (0, -K % BLOCK, 0, -R % rows))
    b = p.view(*v.shape[:-2], p.shape[-2] // rows, rows, p.shape[-1] // BLOCK, BLOCK)
    s = (b.abs().amax(dim=(-3, -1)) / 448).clamp_min(2.0 ** -126).float()
    q = (b / s.double()[..., :, None, :, None]).clamp(-448, 448).float().to(F8)
    q = q.view(torch.uint8).reshape(p.shape)[..., :R, :K].contiguous().view(F8)
    return q, s


def matmul(aq, as_, wq, ws):
    """(out fp64, bound of the fp32 result's error).

    The products of two codes are exact in fp32.  A block's sum takes at most 128
    additions, each off by at most one fp32 step 2^-23 of the magnitudes' sum
    (rounded or cut off); the scale product, the multiply-add of each block and
    the store round once each: (128 + blocks / 2 + 2) * 2^-23 * sum |terms|."""
    a, w = a_values(aq, as_), w_values(wq, ws)
    nk = -(-aq.shape[-1] // BLOCK)
    out = a @ w.transpose(-1, -2)
    mag = a.abs() @ w.abs().transpose(-1, -2)
    return out, (128 + nk / 2 + 2) * 2.0 ** -23 * mag + 1e-37


def quantised_h(h, eh):
    """The values h is rounded to (one scale per 128 columns), and how far a kernel's
    may be from them when its h is within eh: the codes of h - eh and h + eh (a
    value next to a border may land on either side), and the scale's own relative
    error (eh of the block's largest, the division and the rounding)."""
    T, I = h.shape
    top = h.abs().view(T, -1, BLOCK).amax(-1)
    c = (top / 448).clamp_min(2.0 ** -126)
    ce = (eh.view(T, -1, BLOCK).amax(-1) / top.clamp_min(1e-300) + 4 * U32).clamp_max(1.0)
    cw, cew = spread(c, I, 1), spread(ce, I, 1)
    q = e4m3_round(h / cw)
    wide = eh + h.abs() * (cew + 4 * U32)
    lo, hi = e4m3_round((h - wide) / cw), e4m3_round((h + wide) / cw)
    off = torch.maximum((lo - q).abs(), (hi - q).abs()) * cw
    return q * cw, off + (q * cw).abs() * cew


def silu_mul(g, u, eg, eu):
    """silu(g) u and its error bound: |silu'| <= 1.1; the fp32 exponential (2 ulp), the
    division and the two products: 8 half-steps; expf's relative error grows with
    |g| only through the rounding of its argument, which is g itself."""
    sg = g * torch.sigmoid(g)
    h = sg * u
    return h, 1.1 * eg * u.abs() + sg.abs() * eu + 1.1 * eg * eu + h.abs() * 8 * 2.0 ** -23 + 1e-37


def expert_ffn(dims, t, xq, xs, ids, w, residual):
    """(out fp64, bound) of the expert FFN; t: codes and scales by name."""
    E, k, S = dims.n_experts, dims.top_k, dims.n_shared
    T, H = xq.shape
    out = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    ids, w = ids.cpu(), w.cpu().double()
    for e in range(E + S):
        if e < E:
            at = torch.nonzero(ids == e)
            rows, wt = at[:, 0], w[at[:, 0], at[:, 1]]
        else:
            rows, wt = torch.arange(T), torch.ones(T, dtype=torch.float64)
        if rows.numel() == 0:
            continue
        g, eg = matmul(xq[rows], xs[rows], t["gate_q"][e], t["gate_s"][e])
        u, eu = matmul(xq[rows], xs[rows], t["up_q"][e], t["up_s"][e])
        hq, eh = quantised_h(*silu_mul(g, u, eg, eu))
        wd = w_values(t["down_q"][e], t["down_s"][e])
        y = hq @ wd.t()
        m = hq.abs() @ wd.abs().t()
        ey = eh @ wd.abs().t() + (128 + dims.inter / BLOCK / 2 + 2) * 2.0 ** -23 * m
        out.index_add_(0, rows, wt[:, None] * y)
        bound.index_add_(0, rows, wt.abs()[:, None] * ey)
        mag.index_add_(0, rows, wt.abs()[:, None] * y.abs())
    if residual is not None:
        r = residual.cpu().double()
        out += r
        mag += r.abs()
    # the combine: one fp32 rounding per slot; the store: half a bf16 step
    bound = bound + (k + S + 1) * 2.0 ** -23 * mag
    return out, bound + UBF16 * (out.abs() + bound)


def union(ids: torch.Tensor, E: int):
    """The arrays coli_moe_union writes, for a device batch (through the library)."""
    import int4_routed_expert_renorm_b200 as cm
    P = ids.numel()
    new = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    r = (new(min(E, P)), new(1), new(min(E, P) + 1), new(P), new(P))
    cm.coli_moe_union(ids, E, *r)
    return r


def balance(logits, bias, ids, mask, grad_loss, w, d_w):
    """Counts, live tokens, mean probabilities, loss, d_logits, d_bias in fp64 from
    the fp32 routed logits."""
    l32 = logits if bias is None else logits + bias
    l = l32.double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -float("inf")), l)
    T, E = l.shape
    k = ids.shape[1]
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    top = l.amax(1, keepdim=True) if T else l
    e = torch.where(l == top, torch.ones_like(l), torch.exp(l - torch.where(torch.isfinite(top), top, torch.zeros_like(top))))
    e = torch.where(torch.isposinf(top) & (l != top), torch.zeros_like(e), e)
    e = torch.where(torch.isneginf(top), torch.zeros_like(e), e)
    p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    n = int(live.sum())
    li = ids[live].reshape(-1).long()
    li = li[(li >= 0) & (li < E)]
    counts = torch.bincount(li, minlength=E)
    f = counts.double() / max(n * k, 1)
    P = p[live].sum(0) / max(n, 1)
    d = torch.zeros(T, E, dtype=torch.float64)
    if n and grad_loss is not None:
        d += float(grad_loss) * E / n * p * (f[None] - (p * f[None]).sum(1, keepdim=True))
    if d_w is not None:
        wd, dd = w.double(), d_w.double()
        sel = wd * (dd - (wd * dd).sum(1, keepdim=True))
        for j in range(k):
            for t in range(T):
                if 0 <= int(ids[t, j]) < E:
                    d[t, int(ids[t, j])] += sel[t, j]
    d[~live] = 0
    return counts, n, P, float(E * (f * P).sum()), d, d.sum(0)
