"""The router's balance loss, its counts and its gradients against a plain
64-bit statement, at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

from tests import _fp8 as ref
from tests._gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
U = ref.U32


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    return m


def _inputs(T, E, k, seed, bias=True, live=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = 2 * torch.randn(T, E, generator=g)
    b = torch.randn(E, generator=g) if bias else None
    routed = logits + (b if bias else 0)
    top, ids = torch.topk(routed, k, dim=1) if T else (torch.zeros(0, k), torch.zeros(0, k, dtype=torch.int64))
    w = torch.softmax(top, dim=1)
    mask = None
    if live < 1:
        mask = (torch.rand(T, generator=g) < live).to(torch.uint8)
    d_w = torch.randn(T, k, generator=g) / max(T, 1)
    grad = torch.tensor([0.37])
    return logits, b, ids.to(torch.int32), mask, grad, w, d_w


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _run(cm, logits, b, ids, mask, grad, w, d_w, want_bias=True, stream=None):
    T, E = logits.shape
    L, B, I, M, G, W, D = _cuda(logits, b, ids, mask, grad, w, d_w)
    new = lambda *s, dtype=torch.float32: torch.full(s, 77, dtype=dtype, device="cuda")  # noqa: E731
    counts, n, P, loss = new(E, dtype=torch.int32), new(1, dtype=torch.int32), new(E), new(1)
    d, db = new(T, E), new(E) if want_bias else None
    ws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_balance(L, B, I, M, counts, n, P, loss, ws)
    cm.coli_moe_balance_backward(L, B, M, counts, n, G, I, W, D, d, db, ws)
    torch.cuda.synchronize()
    return counts.cpu(), int(n.cpu()), P.cpu().double(), float(loss.cpu()), d.cpu().double(), None if db is None else db.cpu().double()


def _check(got, logits, b, ids, mask, grad, w, d_w):
    """Bounds: p is off by 2 ulp of the exponential, half a step for its argument
    (|l - max| * 2^-24), up to 40 additions of the row sum and a division: (64 +
    |l - max|) half-steps.  Column sums add one half-step per addition along the
    longest chain: a warp's tokens, 8 warps, 296 blocks."""
    want = ref.balance(logits, b, ids, mask, grad, w, d_w)
    counts, n, P, loss, d, db = got
    T, E = logits.shape
    assert torch.equal(counts.long(), want[0]) and n == want[1]
    l = (logits if b is None else logits + b).double()
    gap = (l.amax(1, keepdim=True) - l) if T else l
    gap = torch.where(torch.isfinite(gap), gap, torch.zeros_like(gap)).clamp_max(104.0)
    rel = (64 + gap) * U
    worst = float(rel.max()) if T else 0.0
    chain = -(-T // 2368) + 8 + 296
    assert (P - want[2]).abs().le((worst + (chain + 4) * U) * want[2] + 1e-37).all()
    assert abs(loss - want[3]) <= (worst + (chain + 8) * U) * want[3] + 1e-37
    k = ids.shape[1]
    f = want[0].double() / max(n * k, 1)
    fc = f - 1.0 / E
    p = torch.softmax(torch.nan_to_num(l, nan=-float("inf"), posinf=3e38), 1) if T else l
    p = torch.nan_to_num(p)
    spf = (p * fc.abs()).sum(1, keepdim=True)
    g = 0.0 if grad is None else abs(float(grad))
    off = g * E / max(n, 1) * p * ((rel + 6 * U) * (f - (p * f).sum(1, keepdim=True)).abs() + 4 * U * fc.abs()
                                   + (worst + 48 * U) * spf)
    if d_w is not None:
        wd, dd = w.double(), d_w.double()
        sel = (k + 8) * U * wd * (dd.abs() + (wd * dd).abs().sum(1, keepdim=True))
        for j in range(k):
            at = ids[:, j:j + 1].long()
            fine = (at >= 0) & (at < E)
            off.scatter_add_(1, at.clamp(0, E - 1), torch.where(fine, sel[:, j:j + 1], torch.zeros_like(sel[:, :1])))
    off = off + 2 * U * want[4].abs() + 1e-37
    assert (d - want[4]).abs().le(off).all(), ((d - want[4]).abs() / off).max()
    if db is not None:
        off_b = off.sum(0) + (chain + 2) * U * want[4].abs().sum(0) + 1e-37
        assert (db - want[5]).abs().le(off_b).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (1, 256, 8), (3, 5, 2), (7, 33, 4), (64, 256, 8), (65, 130, 6),
                                   (300, 1024, 32), (257, 1023, 9), (1000, 160, 6), (5003, 64, 4)])
def test_sizes(cm, T, E, k):
    x = _inputs(T, E, k, T + E)
    _check(_run(cm, *x), *x)


@pytest.mark.parametrize("live", [0.5, 0.02])
def test_padded_tokens(cm, live):
    x = _inputs(333, 96, 4, 5, live=live)
    got = _run(cm, *x)
    _check(got, *x)
    assert (got[4][x[3] == 0] == 0).all()


def test_masked_rows_are_not_looked_at(cm):
    logits, b, ids, mask, grad, w, d_w = _inputs(40, 16, 2, 6, live=0.5)
    mask[:2] = torch.tensor([1, 0], dtype=torch.uint8)
    spoilt, bad_ids, bad_w = logits.clone(), ids.clone(), w.clone()
    spoilt[mask == 0] = float("nan")
    bad_ids[mask == 0] = 1 << 30
    bad_w[mask == 0] = float("nan")
    cm.coli_moe_get_status()
    a = _run(cm, logits, b, ids, mask, grad, w, d_w)
    c = _run(cm, spoilt, b, bad_ids, mask, grad, bad_w, d_w)
    assert cm.coli_moe_get_status() == (0, 0)
    assert torch.equal(a[0], c[0]) and a[1] == c[1] and torch.equal(a[2], c[2]) and a[3] == c[3]
    assert torch.equal(a[4], c[4]) and torch.equal(a[5], c[5])


def test_nothing_live(cm):
    logits, b, ids, _, grad, w, d_w = _inputs(20, 16, 2, 7)
    mask = torch.zeros(20, dtype=torch.uint8)
    counts, n, P, loss, d, db = _run(cm, logits, b, ids, mask, grad, w, d_w)
    assert n == 0 and loss == 0 and not counts.any() and not P.any() and not d.any() and not db.any()


def test_empty_batch(cm):
    x = _inputs(0, 16, 2, 8)
    counts, n, P, loss, d, db = _run(cm, *x)
    assert n == 0 and loss == 0 and not counts.any() and not P.any() and not db.any()


def test_without_bias_and_without_a_weight_gradient(cm):
    logits, _, ids, mask, grad, w, _ = _inputs(100, 40, 3, 9, bias=False)
    x = (logits, None, ids, mask, grad, w, None)
    _check(_run(cm, *x), *x)
    logits, b, ids, mask, _, w, d_w = _inputs(100, 40, 3, 10)
    x = (logits, b, ids, mask, None, w, d_w)
    _check(_run(cm, *x, want_bias=False), *x)


def test_masked_experts_and_non_finite_logits(cm):
    """-inf logits get no probability and no gradient; NaN counts as -inf, +inf takes
    the row; a row of -inf has p = 0.  The last two set the status flag."""
    x = list(_inputs(50, 24, 2, 11, bias=False))
    x[0][:, 5] = -float("inf")
    cm.coli_moe_get_status()
    got = _run(cm, *x)
    _check(got, *x)
    assert (got[4][:, 5][(x[2] != 5).all(1)] == 0).all()      # where its weight was not selected either
    assert cm.coli_moe_get_status() == (0, 0)
    x[0][3, :] = -float("inf")
    x[0][4, 7] = float("nan")
    x[0][6, 2] = float("inf")
    x[0][6, 9] = float("inf")
    got = _run(cm, *x)
    want = ref.balance(*x)
    assert torch.isfinite(got[4]).all()
    assert torch.allclose(got[4], want[4], rtol=1e-4, atol=1e-6) and abs(got[3] - want[3]) < 1e-5
    st, flags = cm.coli_moe_get_status()
    assert flags == cm._lib.COLI_FLAG_NONFINITE
    # the type's lowest value as a mask, in whole rows too: uniform over the row
    y = list(_inputs(6, 8, 2, 12, bias=False))
    y[0][:, :] = torch.finfo(torch.float32).min
    y[0][1, 3] = 0.0
    got, want = _run(cm, *y), ref.balance(*y)
    assert torch.allclose(got[4], want[4], rtol=1e-4, atol=1e-7) and torch.allclose(got[2], want[2], rtol=1e-5)


def test_ids_out_of_range_and_repeated(cm):
    logits, b, ids, mask, grad, w, d_w = _inputs(30, 12, 3, 13)
    ids[0, 0], ids[1, 1], ids[2, 2] = -1, 12, 1 << 30
    ids[5, 0] = ids[5, 1] = ids[5, 2] = 4        # the same expert three times
    cm.coli_moe_get_status()
    got = _run(cm, logits, b, ids, mask, grad, w, d_w)
    st, flags = cm.coli_moe_get_status()
    assert flags == cm._lib.COLI_FLAG_BAD_ID
    _check(got, logits, b, ids, mask, grad, w, d_w)


def test_gradient_against_differences(cm):
    """The loss with its counts held, differentiated numerically in 64 bits."""
    logits, b, ids, mask, grad, w, _ = _inputs(9, 10, 2, 14, live=0.7)
    mask[0] = 1
    _, _, _, _, d, db = _run(cm, logits, b, ids, mask, torch.tensor([1.0]), w, None)
    live = mask.bool()
    n, E, k = int(live.sum()), 10, 2
    f = torch.bincount(ids[live].reshape(-1).long(), minlength=E).double() / (n * k)

    def loss(l):
        return E * (f * torch.softmax(l, 1)[live].mean(0)).sum()

    l0, eps = (logits + b).double(), 1e-5
    for t, e in ((0, 0), (3, 7), (8, 9), (5, 2)):
        hi, lo = l0.clone(), l0.clone()
        hi[t, e] += eps
        lo[t, e] -= eps
        num = (loss(hi) - loss(lo)) / (2 * eps)
        # central differences: eps^2 and 2^-52 / eps; the kernel: about 100 half-steps of a value below 1
        assert abs(float(num) - float(d[t, e])) <= 1e-5 * abs(float(num)) + 1e-7
    auto = l0.clone().requires_grad_(True)
    loss(auto).backward()
    assert torch.allclose(db, auto.grad.sum(0), rtol=1e-5, atol=1e-7)


def test_weight_gradient_against_differences(cm):
    logits, b, ids, _, _, w, d_w = _inputs(6, 12, 3, 15)
    got = _run(cm, logits, b, ids, None, None, w, d_w)
    l = (logits + b).double().requires_grad_(True)
    wt = torch.softmax(torch.gather(l, 1, ids.long()), 1)
    (wt * d_w.double()).sum().backward()
    assert torch.allclose(got[4], l.grad, rtol=1e-5, atol=1e-8)


def test_same_bits_every_time_and_captured(cm):
    """No atomics on floats: the same bits each call; and replayed from a graph on
    another stream, with new inputs in the same buffers."""
    T, E, k = 700, 160, 6
    x = _inputs(T, E, k, 16, live=0.9)
    first = _run(cm, *x)
    for _ in range(3):
        again = _run(cm, *x)
        assert all(torch.equal(a, c) if isinstance(a, torch.Tensor) else a == c for a, c in zip(first, again))
    L, B, I, M, G, W, D = _cuda(*x)
    new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    out = (new(E, dtype=torch.int32), new(1, dtype=torch.int32), new(E), new(1), new(T, E), new(E))
    ws = [torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        cm.coli_moe_balance(L, B, I, M, *out[:4], ws[0])
        cm.coli_moe_balance_backward(L, B, M, out[0], out[1], G, I, W, D, out[4], out[5], ws[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[4].cpu().double(), first[4]) and torch.equal(out[5].cpu().double(), first[5])
    y = _inputs(T, E, k, 17, live=0.9)
    for dst, src in zip((L, B, I, M, G, W, D), y):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    got = (out[0].cpu(), int(out[1]), out[2].cpu().double(), float(out[3]), out[4].cpu().double(), out[5].cpu().double())
    _check(got, *y)


def test_counts_feed_a_usage_profile(cm):
    """The counts of a routed batch are what the tier's usage profile counts."""
    T, E, k = 37, 16, 2
    logits, b, *_ = _inputs(T, E, k, 18)
    L, B = logits.cuda(), b.cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    cm.coli_moe_route(L, B, ids, w)
    counts, n = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    P, loss = torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_balance(L, B, ids, None, counts, n, P, loss, ws)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.cpu().numpy().reshape(-1), minlength=E))
    assert int(counts.sum()) == T * k and abs(float(P.sum()) - 1) < 1e-5


def test_unaligned_rows_and_in_place_gradient(cm):
    """E a multiple of 4 with rows that start off a 16-byte boundary; d_logits in
    place of the logits."""
    T, E, k = 50, 64, 4
    logits, b, ids, mask, grad, w, d_w = x = _inputs(T, E, k, 19)
    buf = torch.zeros(T * E + 3, device="cuda")
    L = buf[3:].view(T, E)
    L.copy_(logits)
    B, I, G, W, D = _cuda(b, ids, grad, w, d_w)
    out = (torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"),
           torch.empty(E, device="cuda"), torch.empty(1, device="cuda"))
    db = torch.empty(E, device="cuda")
    ws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_balance(L, B, I, None, *out, ws)
    cm.coli_moe_balance_backward(L, B, None, out[0], out[1], G, I, W, D, L, db, ws)
    torch.cuda.synchronize()
    _check((out[0].cpu(), int(out[1]), out[2].cpu().double(), float(out[3]), L.cpu().double(), db.cpu().double()), *x)


@pytest.mark.parametrize("T", [255, 256, 257, 4096, 4737])
def test_one_and_two_launches(cm, T):
    """Up to 256 tokens one launch does everything, more take a second pass; 4736
    tokens are one per warp."""
    x = _inputs(T, 40, 3, T, live=0.9)
    _check(_run(cm, *x), *x)


def test_offsets_past_32_bits(cm):
    """2.3e9 logits: the counts and the mean exactly as far as integers go, and rows
    of the gradient from both ends."""
    T, E, k = 2_200_003, 1024, 2
    g = torch.Generator(device="cuda").manual_seed(60)
    logits = torch.randn(T, E, device="cuda", generator=g)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=g)
    new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    counts, n, P, loss = new(E, dtype=torch.int32), new(1, dtype=torch.int32), new(E), new(1)
    ws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_balance(logits, None, ids, None, counts, n, P, loss, ws)
    assert torch.equal(counts.long(), torch.bincount(ids.reshape(-1).long(), minlength=E)) and int(n) == T
    assert abs(float(P.double().sum()) - 1) < 1e-4
    grad = torch.ones(1, device="cuda")
    rows = torch.tensor([0, 1, 2_097_151, 2_097_152, 2_200_002]).cuda()
    l = logits[rows].double().cpu()
    cm.coli_moe_balance_backward(logits, None, None, counts, n, grad, ids, None, None, logits, None, ws)
    p = torch.softmax(l, 1)
    f = counts.cpu().double() / (T * k)
    want = E / T * p * (f - (p * f).sum(1, keepdim=True))
    # as in _check, with |l - max| below 16: 80 half-steps of p, the rest of f and its sum
    fc = (f - 1.0 / E).abs()
    off = E / T * p * ((86 * U) * (f - (p * f).sum(1, keepdim=True)).abs() + 4 * U * fc + 128 * U * (p * fc).sum(1, keepdim=True))
    assert (logits[rows].cpu().double() - want).abs().le(off + 2 * U * want.abs() + 1e-37).all()
