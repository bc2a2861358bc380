"""Refusals of the balance loss and the 8-bit floating-point operators: the C
entries' argument checks and the binding's.  CPU only: no call reaches a launch."""
import ctypes

import pytest
import torch

A = 0x10000      # a made-up aligned address; no call below gets as far as using it


@pytest.fixture(scope="module")
def cm():
    from int4_routed_expert_renorm_b200.build import build
    build()
    import int4_routed_expert_renorm_b200 as m
    return m


@pytest.fixture(scope="module")
def lib(cm):
    return cm._lib._lib


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _balance(lib, T=4, E=16, k=2, logits=A, ids=A, counts=A, n=A, P=A, loss=A, ws=A, size=1 << 30):
    return lib.coli_moe_balance(logits, None, ids, None, T, E, k, counts, n, P, loss, ws, size, None)


def test_balance_refusals(cm, lib):
    assert _balance(lib, T=-1) == INVALID and _balance(lib, E=0) == INVALID and _balance(lib, k=0) == INVALID
    assert _balance(lib, E=1025) == UNSUPPORTED and _balance(lib, E=64, k=33) == UNSUPPORTED
    assert _balance(lib, E=4, k=5) == UNSUPPORTED and _balance(lib, T=(1 << 23) + 1) == UNSUPPORTED
    for name in ("logits", "ids", "counts", "n", "P", "loss", "ws"):
        assert _balance(lib, **{name: None}) == INVALID, name
    assert _balance(lib, ws=A + 64) == INVALID
    need = cm.coli_moe_balance_workspace_bytes(4, 16)
    assert need > 0 and _balance(lib, size=need - 1) == WORKSPACE
    assert cm.coli_moe_balance_workspace_bytes(-1, 16) == 0 and cm.coli_moe_balance_workspace_bytes(4, 1025) == 0
    assert cm.coli_moe_balance_workspace_bytes(4, 0) == 0 and cm.coli_moe_balance_workspace_bytes(0, 4) > 0
    sizes = [cm.coli_moe_balance_workspace_bytes(t, 256) for t in (0, 1, 8, 9, 100, 5000, 1 << 20)]
    assert sizes == sorted(sizes)


def _backward(lib, T=4, E=16, k=2, logits=A, counts=A, n=A, grad=A, ids=A, w=A, dw=A, d=A, ws=A, size=1 << 30):
    return lib.coli_moe_balance_backward(logits, None, None, counts, n, grad, ids, w, dw, T, E, k, d, None, ws, size, None)


def test_balance_backward_refusals(cm, lib):
    assert _backward(lib, T=-1) == INVALID and _backward(lib, E=2000) == UNSUPPORTED
    for name in ("logits", "counts", "n", "ids", "w", "d", "ws"):
        assert _backward(lib, **{name: None}) == INVALID, name
    assert _backward(lib, grad=None, dw=None) == INVALID
    assert _backward(lib, size=16) == WORKSPACE


def _norm(lib, x=A, r=None, w=None, eps=1e-6, T=2, H=256, s=None, n=None, q=A, sc=A):
    return lib.coli_add_rmsnorm_fp8(x, r, w, eps, T, H, s, n, q, sc, None)


def test_norm_refusals(lib):
    assert _norm(lib, T=0) == OK
    assert _norm(lib, T=-1) == INVALID and _norm(lib, H=0) == INVALID
    assert _norm(lib, eps=-1.0) == INVALID and _norm(lib, eps=float("nan")) == INVALID
    assert _norm(lib, H=200) == UNSUPPORTED and _norm(lib, H=32768 + 128) == UNSUPPORTED
    for name in ("x", "q", "sc"):
        assert _norm(lib, **{name: None}) == INVALID, name
    for name in ("x", "r", "w", "s", "n", "q"):
        assert _norm(lib, **{name: A + 8}) == INVALID, name
    B = A + 4096
    assert _norm(lib, n=A) == INVALID and _norm(lib, r=B, n=B) == INVALID and _norm(lib, s=B, n=B) == INVALID


def _matmul(lib, a=A, as_=A, w=A, ws=A, M=4, N=64, K=256, out=A, flags=0):
    return lib.coli_fp8_matmul(a, as_, w, ws, M, N, K, out, flags, None)


def test_matmul_refusals(lib):
    assert _matmul(lib, M=0) == OK
    assert _matmul(lib, M=-1) == INVALID and _matmul(lib, N=0) == INVALID and _matmul(lib, K=0) == INVALID
    assert _matmul(lib, flags=2) == INVALID
    assert _matmul(lib, K=100) == UNSUPPORTED and _matmul(lib, K=8) == UNSUPPORTED
    assert _matmul(lib, K=(1 << 20) + 16) == UNSUPPORTED and _matmul(lib, N=(1 << 21) + 1) == UNSUPPORTED
    assert _matmul(lib, M=(1 << 24) + 1) == UNSUPPORTED
    for name in ("a", "as_", "w", "ws", "out"):
        assert _matmul(lib, **{name: None}) == INVALID, name
    for name in ("a", "w", "out"):
        assert _matmul(lib, **{name: A + 8}) == INVALID, name
    assert _matmul(lib, as_=A + 2) == INVALID and _matmul(lib, ws=A + 1) == INVALID


def _ffn(cm, lib, T=4, size=1 << 40, weights=None, **kw):
    d = dict(hidden=256, inter=128, n_experts=8, top_k=2, n_shared=1, group=128, code_bits=8)
    args = dict(x=A, xs=A, ids=A, w=A, u=A, nu=A, seg=A, perm=A, pos=A, out=A, ws=A, res=None)
    for name, v in kw.items():
        (d if name in d else args)[name] = v
    dims = cm.coli_moe_dims(**d)
    weights = cm.coli_moe_weights_fp8(*[A] * 6) if weights is None else weights
    g = args
    return lib.coli_moe_expert_ffn_fp8(ctypes.byref(dims), ctypes.byref(weights), g["x"], g["xs"], T, g["ids"], g["w"],
                                       g["u"], g["nu"], g["seg"], g["perm"], g["pos"], g["res"], g["out"], g["ws"], size,
                                       None)


def test_expert_ffn_refusals(cm, lib):
    assert _ffn(cm, lib, T=0) == OK and _ffn(cm, lib, T=-1) == INVALID
    for bad in (dict(group=32), dict(group=64), dict(code_bits=4), dict(hidden=200), dict(inter=64), dict(hidden=0),
                dict(n_experts=1025), dict(n_experts=0), dict(top_k=0), dict(top_k=9), dict(n_shared=5),
                dict(n_shared=-1), dict(n_experts=64, top_k=33), dict(hidden=1 << 27)):
        assert _ffn(cm, lib, **bad) == UNSUPPORTED, bad
    assert _ffn(cm, lib, T=1 << 23) == UNSUPPORTED
    for name in ("x", "xs", "ids", "w", "u", "nu", "seg", "perm", "pos", "out", "ws"):
        assert _ffn(cm, lib, **{name: None}) == INVALID, name
    for name in ("x", "out", "res", "ws"):
        assert _ffn(cm, lib, **{name: A + 8}) == INVALID, name
    for i in range(6):
        ptrs = [A] * 6
        ptrs[i] = None
        assert _ffn(cm, lib, weights=cm.coli_moe_weights_fp8(*ptrs)) == INVALID, i
        ptrs[i] = A + 4
        assert _ffn(cm, lib, weights=cm.coli_moe_weights_fp8(*ptrs)) == INVALID, i
    dims = cm.dims_for(256, 128, 8, 2, 1, group=128, code_bits=8)
    need = cm.coli_moe_fp8_workspace_bytes(dims, 4)
    assert need > 0 and _ffn(cm, lib, size=need - 1) == WORKSPACE
    assert cm.coli_moe_fp8_workspace_bytes(cm.dims_for(256, 128, 8, 2, 1), 4) == 0
    assert cm.coli_moe_fp8_workspace_bytes(dims, -1) == 0 and cm.coli_moe_fp8_workspace_bytes(dims, 0) > 0
    sizes = [cm.coli_moe_fp8_workspace_bytes(dims, t) for t in range(0, 300, 7)]
    assert sizes == sorted(sizes)


def test_integer_containers_still_refuse_these_dims(cm):
    """The 8-bit floating-point dims are not dims of the integer calls."""
    assert cm.coli_moe_workspace_bytes(cm.dims_for(6144, 2048, 256, 8, 1, group=128, code_bits=8), 4) == 0


def test_binding_refuses_host_strided_short_and_mistyped_tensors(cm):
    f = torch.float32
    logits, ids, i1, e, ws = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), \
        torch.zeros(16), torch.zeros(1 << 20, dtype=torch.uint8)
    counts, loss = torch.zeros(16, dtype=torch.int32), torch.zeros(1)
    good = dict(logits=logits, bias=e, topk_ids=ids, mask=None, counts=counts, n_live=i1, prob_mean=e, loss=loss, ws=ws)
    with pytest.raises(ValueError, match="device memory"):
        cm.coli_moe_balance(**good)
    for name, bad, say in (("bias", torch.zeros(15), "bias"), ("topk_ids", ids.long(), "topk_ids"),
                           ("topk_ids", torch.zeros(3, 2, dtype=torch.int32), "topk_ids"),
                           ("mask", torch.zeros(4), "mask"), ("mask", torch.zeros(3, dtype=torch.uint8), "mask"),
                           ("counts", torch.zeros(16), "counts"), ("loss", torch.zeros(2), "loss"),
                           ("logits", logits.int(), "logits"), ("logits", logits[0], "logits")):
        with pytest.raises(ValueError, match=say):
            cm.coli_moe_balance(**{**good, name: bad})
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    q, sc = torch.zeros(2, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 2)
    for kw, say in ((dict(x=x.half()), "x"), (dict(residual=x[:1]), "residual"), (dict(weight=x[0, :9]), "weight"),
                    (dict(q=q.view(torch.float8_e5m2)), "q"), (dict(q_scale=sc[:1]), "q_scale"),
                    (dict(norm_out=x.float()), "norm_out"), (dict(), "device memory"), (dict(x=x[0]), "two dimensions")):
        a = {**dict(x=x, residual=None, weight=None, eps=1e-6, sum_out=None, norm_out=None, q=q, q_scale=sc), **kw}
        with pytest.raises(ValueError, match=say):
            cm.coli_add_rmsnorm_fp8(**a)
    a, w = torch.zeros(3, 256, dtype=torch.float8_e4m3fn), torch.zeros(130, 256, dtype=torch.float8_e4m3fn)
    good = dict(a=a, a_scale=torch.zeros(3, 2), w=w, w_scale=torch.zeros(2, 2), out=torch.zeros(3, 130))
    for kw, say in ((dict(w=w[:, :128]), "w"), (dict(w_scale=torch.zeros(1, 2)), "w_scale"), (dict(a_scale=sc), "a_scale"),
                    (dict(out=torch.zeros(3, 129)), "out"), (dict(out=torch.zeros(3, 130, dtype=torch.float16)), "out"),
                    (dict(out=torch.zeros(3, 130, dtype=torch.float64)), "out"), (dict(), "device memory")):
        with pytest.raises(ValueError, match=say):
            cm.coli_fp8_matmul(**{**good, **kw})
    with pytest.raises(ValueError, match="contiguous"):
        cm.coli_fp8_matmul(**{**good, "a": torch.zeros(256, 3, dtype=torch.float8_e4m3fn).t(),
                              "a_scale": torch.zeros(3, 2)})


def test_holder_refuses_wrong_shapes(cm):
    t = {n: torch.zeros(s, dtype=torch.uint8 if n[-1] == "q" else torch.float32)
         for n, s in (("gate_q", (5, 128, 256)), ("up_q", (5, 128, 256)), ("down_q", (5, 256, 128)),
                      ("gate_s", (5, 1, 2)), ("up_s", (5, 1, 2)), ("down_s", (5, 2, 1)))}
    with pytest.raises(ValueError, match="device memory"):
        cm.fp8_weights(**t)
    with pytest.raises(ValueError, match="down_q"):
        cm.fp8_weights(**{**t, "down_q": torch.zeros(5, 128, 256, dtype=torch.uint8)})
    with pytest.raises(ValueError, match="up_s"):
        cm.fp8_weights(**{**t, "up_s": torch.zeros(5, 1, 3)})
    with pytest.raises(ValueError, match="gate_q"):
        cm.Fp8MoELayer(cm.dims_for(256, 128, 8, 2, 1, group=128, code_bits=8), t)
