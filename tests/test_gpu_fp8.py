"""The 8-bit floating-point operators against plain 64-bit statements: the norm
with its 8-bit rows, the block-scaled product, the expert FFN, and a run of them
together with Route, Union and the balance loss."""
import pytest
import torch

from tests import _fp8 as ref
from tests._gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
U = ref.U32
F8 = ref.F8


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    return m


# ------------------------------------------------------------------- norm --

def _norm_check(cm, x, r, w, eps=1e-6, in_place=None, want_norm=True):
    """Bounds: the sum is one bf16 rounding of an exact fp32 sum (equal).  n: the row's
    sum of squares takes at most 8 * 16 + 8 additions per path, the mean, the root,
    its inverse and two products a few more: relative (160 / 2 + 8) half-steps.  The
    scale adds a division; a code may fall on either side of a border when n is
    within that of it."""
    T, H = x.shape
    X, R, W = (None if t is None else t.cuda() for t in (x, r, w))
    s_out = torch.empty_like(X) if in_place is None else {"x": X, "r": R}[in_place]
    n_out = torch.empty_like(X) if want_norm else None
    q = torch.empty(T, H, dtype=F8, device="cuda")
    sc = torch.empty(T, H // 128, device="cuda")
    cm.coli_add_rmsnorm_fp8(X, R, W, eps, s_out, n_out, q, sc)
    torch.cuda.synchronize()
    s = (x.float() + (0 if r is None else r.float())).to(torch.bfloat16)
    assert torch.equal(s_out.cpu(), s)
    v = s.double()
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    rel = 88 * U
    if want_norm:
        assert (n_out.cpu().double() - n).abs().le((rel + ref.UBF16) * n.abs() + 1e-37).all()
    top = n.abs().view(T, -1, 128).amax(-1)
    c = (top / 448).clamp_min(2.0 ** -126)
    assert (sc.cpu().double() - c).abs().le((rel + 2 * U) * c).all()
    cw = ref.spread(c, H, 1)
    got = ref.decode(q)
    lo, hi = ref.e4m3_round(n / cw * (1 - 2 * rel - 4 * U)), ref.e4m3_round(n / cw * (1 + 2 * rel + 4 * U))
    assert ((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all()
    return q, sc


@pytest.mark.parametrize("T,H", [(1, 128), (1, 6144), (2, 256), (3, 2176), (5, 2048), (17, 4096), (4, 8192), (3, 16384),
                                 (2, 32768), (333, 640)])
@pytest.mark.parametrize("res,wt", [(True, True), (False, False), (True, False)])
def test_norm(cm, T, H, res, wt):
    g = torch.Generator().manual_seed(T * 7 + H)
    x = (3 * torch.randn(T, H, generator=g)).to(torch.bfloat16)
    r = torch.randn(T, H, generator=g).to(torch.bfloat16) if res else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16) if wt else None
    _norm_check(cm, x, r, w)


def test_norm_in_place_and_without_its_bf16_copy(cm):
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(9, 384, generator=g).to(torch.bfloat16) for _ in range(2))
    _norm_check(cm, x, r, None, in_place="x")
    _norm_check(cm, x, r, None, in_place="r", want_norm=False)


def test_norm_of_zeros_small_and_large_values(cm):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 512, generator=g)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-18
    x[3] *= 1e15
    x[4, 5] = 1e6           # one loud value: its block's others round to little or nothing
    x[5, :] = 0
    x[5, 511] = 1
    _norm_check(cm, x.to(torch.bfloat16), None, None)
    q, sc = _norm_check(cm, torch.zeros(2, 256, dtype=torch.bfloat16), None, None, eps=1e-6)
    assert not q.view(torch.uint8).any() and (sc == 2.0 ** -126).all()


def test_norm_flags_rows_that_are_not_finite(cm):
    x = torch.ones(3, 256, dtype=torch.bfloat16)
    x[1, 7] = float("nan")
    cm.coli_moe_get_status()
    X = x.cuda()
    q = torch.empty(3, 256, dtype=torch.uint8, device="cuda")
    sc = torch.empty(3, 2, device="cuda")
    cm.coli_add_rmsnorm_fp8(X, None, None, 1e-6, None, None, q, sc)
    st, flags = cm.coli_moe_get_status()
    assert flags == cm._lib.COLI_FLAG_NONFINITE
    assert (q[1] == 0x7F).all() and torch.isnan(sc[1]).all()
    assert torch.isfinite(sc[0]).all() and torch.isfinite(sc[2]).all() and (q[0] == q[2]).all()


# ---------------------------------------------------------------- product --

def _operands(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g, dtype=torch.float64) * torch.exp(torch.randn(M, 1, generator=g, dtype=torch.float64))
    w = torch.randn(N, K, generator=g, dtype=torch.float64) * 0.05
    return (*ref.block_quantise(a, 1), *ref.block_quantise(w, 128))


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (1, 4096, 6144), (2, 640, 2048), (3, 129, 144), (8, 576, 512),
                                   (16, 256, 1024), (17, 384, 384), (33, 1001, 1040), (64, 256, 256), (65, 136, 2064),
                                   (128, 512, 512), (161, 260, 640), (200, 2048, 128), (301, 1001, 1040), (511, 300, 272),
                                   (1000, 1280, 384), (1537, 777, 400)])
@pytest.mark.parametrize("f32", [True, False])
def test_matmul(cm, M, N, K, f32):
    aq, as_, wq, ws = _operands(M, N, K, M + N + K)
    want, bound = ref.matmul(aq, as_, wq, ws)
    pad = 64                                             # rows behind the last one stay as they were
    buf = torch.full((M * N + pad,), 7, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    out = buf[:M * N].view(M, N)
    cm.coli_fp8_matmul(aq.cuda(), as_.cuda(), wq.cuda(), ws.cuda(), out)
    torch.cuda.synchronize()
    assert (buf[M * N:] == 7).all()
    if not f32:
        bound = bound + ref.UBF16 * (want.abs() + bound)
    err = (out.cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())
    assert cm.coli_moe_get_status() == (0, 0)


def test_matmul_rows_do_not_depend_on_the_batch_and_repeat(cm):
    """A row's bits are the same on every call."""
    aq, as_, wq, ws = (t.cuda() for t in _operands(40, 512, 1024, 2))
    outs = []
    for _ in range(3):
        out = torch.empty(40, 512, device="cuda")
        cm.coli_fp8_matmul(aq, as_, wq, ws, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_matmul_nan_codes_stay_in_their_row_and_column(cm):
    aq, as_, wq, ws = _operands(5, 130, 256, 4)
    aq.view(torch.uint8)[2, 9] = 0x7F
    wq.view(torch.uint8)[128, 200] = 0xFF
    out = torch.empty(5, 130, device="cuda")
    cm.coli_fp8_matmul(aq.cuda(), as_.cuda(), wq.cuda(), ws.cuda(), out)
    bad = torch.isnan(out.cpu())
    want = torch.zeros(5, 130, dtype=torch.bool)
    want[2] = True
    want[:, 128] = True
    assert torch.equal(bad, want)


def test_matmul_extreme_scales(cm):
    """Zero scales, and scales far apart from block to block."""
    aq, as_, wq, ws = _operands(20, 300, 640, 5)
    as_[:, 1] = 0
    as_[3] *= 1e-20
    ws[1] *= 1e15
    ws[:, 2] *= 1e-6
    want, bound = ref.matmul(aq, as_, wq, ws)
    out = torch.empty(20, 300, device="cuda")
    cm.coli_fp8_matmul(aq.cuda(), as_.cuda(), wq.cuda(), ws.cuda(), out)
    assert (out.cpu().double() - want).abs().le(bound).all()


def test_matmul_on_a_stream_and_in_a_graph(cm):
    aq, as_, wq, ws = (t.cuda() for t in _operands(50, 640, 768, 6))
    eager = torch.empty(50, 640, device="cuda")
    cm.coli_fp8_matmul(aq, as_, wq, ws, eager)
    out = torch.zeros(50, 640, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        cm.coli_fp8_matmul(aq, as_, wq, ws, out)
    bq, bs, _, _ = (t.cuda() for t in _operands(50, 640, 768, 7))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    aq.copy_(bq)
    as_.copy_(bs)
    graph.replay()
    torch.cuda.synchronize()
    want, bound = ref.matmul(bq.cpu(), bs.cpu(), wq.cpu(), ws.cpu())
    assert (out.cpu().double() - want).abs().le(bound).all()


# -------------------------------------------------------------- expert FFN --

def _experts(E, S, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    t = {}
    for name, R, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        v = torch.randn(E + S, R, K, generator=g, dtype=torch.float64) / K ** 0.5
        t[name + "_q"], t[name + "_s"] = ref.block_quantise(v, 128)
    return t


def _routed(T, E, k, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) - skew * torch.arange(E)
    top, ids = torch.topk(logits, k, dim=1)
    return logits, ids.to(torch.int32), torch.softmax(top, 1)


def _ffn(cm, dims, t, xq, xs, ids, w, residual, out=None, ws=None, arrays=None, stream=None):
    dev = {n: v.cuda() for n, v in t.items()}
    T = xq.shape[0]
    out = torch.full((T, dims.hidden), 3, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = torch.empty(cm.coli_moe_fp8_workspace_bytes(dims, T), dtype=torch.uint8, device="cuda") if ws is None else ws
    arrays = ref.union(ids.cuda(), dims.n_experts) if arrays is None else arrays
    cm.coli_moe_expert_ffn_fp8(dims, cm.fp8_weights(**dev), xq.cuda(), xs.cuda(), ids.cuda(), w.cuda(), *arrays,
                               None if residual is None else residual.cuda(), out, ws, stream)
    torch.cuda.synchronize()
    return out


CASES = [  # T, E, k, S, H, I, skew
    (1, 1, 1, 0, 128, 128, 0.0),
    (1, 4, 2, 1, 256, 128, 0.0),
    (2, 16, 2, 1, 384, 256, 0.0),
    (5, 8, 8, 0, 512, 384, 0.0),
    (8, 64, 8, 1, 1024, 256, 0.0),
    (17, 8, 3, 2, 640, 128, 0.0),
    (33, 4, 1, 4, 256, 384, 0.0),
    (64, 6, 2, 1, 384, 640, 1.0),
    (100, 3, 3, 0, 512, 256, 0.0),
    (161, 5, 1, 1, 256, 256, 4.0),     # nearly every token on one expert: more than one token block
    (400, 9, 4, 1, 256, 128, 0.5),
    (700, 20, 2, 0, 384, 128, 0.2),
]


@pytest.mark.parametrize("T,E,k,S,H,I,skew", CASES)
def test_expert_ffn(cm, T, E, k, S, H, I, skew):
    dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
    t = _experts(E, S, H, I, T)
    g = torch.Generator().manual_seed(T + 1)
    xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
    _, ids, w = _routed(T, E, k, T + 2, skew)
    residual = torch.randn(T, H, generator=g).to(torch.bfloat16) if S != 2 else None
    out = _ffn(cm, dims, t, xq, xs, ids, w, residual)
    want, bound = ref.expert_ffn(dims, t, xq, xs, ids, w, residual)
    err = (out.cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())
    assert cm.coli_moe_get_status() == (0, 0)


def test_expert_ffn_glm_shape_single_token(cm):
    """One token at the GLM-5.2 layer's widths (8 experts of them)."""
    dims = cm.dims_for(6144, 2048, 8, 8, 1, group=128, code_bits=8)
    t = _experts(8, 1, 6144, 2048, 1)
    g = torch.Generator().manual_seed(2)
    xq, xs = ref.block_quantise(torch.randn(1, 6144, generator=g, dtype=torch.float64), 1)
    _, ids, w = _routed(1, 8, 8, 3)
    r = torch.randn(1, 6144, generator=g).to(torch.bfloat16)
    want, bound = ref.expert_ffn(dims, t, xq, xs, ids, w, r)
    out = _ffn(cm, dims, t, xq, xs, ids, w, r)
    err = (out.cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())


def test_expert_ffn_skips_pairs_out_of_range_and_repeats(cm):
    """An id outside [0, E) adds nothing; an expert selected twice by a token counts
    twice; the residual may be the output."""
    T, E, k, H, I = 12, 6, 3, 256, 128
    dims = cm.dims_for(H, I, E, k, 0, group=128, code_bits=8)
    t = _experts(E, 0, H, I, 5)
    g = torch.Generator().manual_seed(6)
    xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
    _, ids, w = _routed(T, E, k, 7)
    ids[0, 1], ids[3, 0], ids[3, 1], ids[3, 2] = -1, 9, -5, 6     # token 3: nothing at all
    ids[4] = 2
    r = torch.randn(T, H, generator=g).to(torch.bfloat16)
    out = r.cuda()
    cm.coli_moe_get_status()
    dev_ids = ids.cuda()
    arrays = ref.union(dev_ids, E)
    assert cm.coli_moe_get_status()[1] == cm._lib.COLI_FLAG_BAD_ID
    dev = {n: v.cuda() for n, v in t.items()}
    ws = torch.empty(cm.coli_moe_fp8_workspace_bytes(dims, T), dtype=torch.uint8, device="cuda")
    cm.coli_moe_expert_ffn_fp8(dims, cm.fp8_weights(**dev), xq.cuda(), xs.cuda(), dev_ids, w.cuda(), *arrays, out, out, ws)
    want, bound = ref.expert_ffn(dims, t, xq, xs, ids, w, r)
    assert (out.cpu().double() - want).abs().le(bound).all()
    assert torch.equal(out.cpu()[3], r[3])
    assert cm.coli_moe_get_status() == (0, 0)


def test_expert_ffn_repeats_bit_for_bit_whatever_the_workspace_holds(cm):
    T, E, k, S, H, I = 70, 8, 2, 1, 512, 256
    dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
    t = _experts(E, S, H, I, 8)
    g = torch.Generator().manual_seed(9)
    xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
    _, ids, w = _routed(T, E, k, 10)
    n = cm.coli_moe_fp8_workspace_bytes(dims, T)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(_ffn(cm, dims, t, xq, xs, ids, w, None, ws=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_calls_at_once_and_captured(cm):
    """Two streams with a workspace each, and a captured call replayed with a new
    routing in the same buffers."""
    T, E, k, S, H, I = 24, 8, 2, 1, 512, 256
    dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
    t = _experts(E, S, H, I, 11)
    dev = {n: v.cuda() for n, v in t.items()}
    weights = cm.fp8_weights(**dev)
    g = torch.Generator().manual_seed(12)
    ins = []
    for i in range(2):
        xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
        _, ids, w = _routed(T, E, k, 13 + i)
        ins.append((xq, xs, ids, w))
    want = [ref.expert_ffn(dims, t, *i, None) for i in ins]
    n = cm.coli_moe_fp8_workspace_bytes(dims, T)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    on_dev = [tuple(v.cuda() for v in i) for i in ins]
    arrays = [ref.union(d[2], E) for d in on_dev]
    torch.cuda.synchronize()
    for _ in range(4):
        for d, a, o, ws, st in zip(on_dev, arrays, outs, wss, streams):
            cm.coli_moe_expert_ffn_fp8(dims, weights, *d, *a, None, o, ws, st)
    torch.cuda.synchronize()
    for o, (v, b) in zip(outs, want):
        assert (o.cpu().double() - v).abs().le(b).all()
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    x, a = on_dev[0], arrays[0]
    with torch.cuda.graph(graph):
        cm.coli_moe_union(x[2], E, *a)
        cm.coli_moe_expert_ffn_fp8(dims, weights, *x, *a, None, out, wss[0])
    for dst, src in zip(x, on_dev[1]):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, outs[1])


# ------------------------------------------------------- a run of them all --

def test_layer_path(cm):
    """norm -> Route -> balance -> Union -> experts -> the next norm, as a layer and the
    head after it use them, through the holder and call by call."""
    T, E, k, S, H, I = 29, 12, 3, 1, 384, 256
    dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
    t = _experts(E, S, H, I, 20)
    dev = {n: v.cuda() for n, v in t.items()}
    g = torch.Generator().manual_seed(21)
    weight = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    layer = cm.Fp8MoELayer(dims, dev, weight)
    x, r = ((torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    logits = torch.randn(T, E, generator=g).cuda()
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ids, w = layer.forward(x, logits, out, layer.workspace(T), residual=r)
    h = torch.empty_like(x)
    q, s = layer.norm(x, r, sum_out=h)
    want, bound = ref.expert_ffn(dims, t, q.cpu(), s.cpu(), ids.cpu(), w.cpu(), h.cpu())
    assert (out.cpu().double() - want).abs().le(bound).all()
    assert torch.equal(ids.cpu(), torch.topk(logits.cpu(), k, dim=1).indices.int())
    # the router's statistics of the same batch, and the head's product over the next norm
    counts, n = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    P, loss = torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    bws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_balance(logits, None, ids, None, counts, n, P, loss, bws)
    assert torch.equal(counts.cpu().long(), torch.bincount(ids.cpu().reshape(-1).long(), minlength=E))
    head_q, head_s = ref.block_quantise(torch.randn(200, H, generator=g, dtype=torch.float64) * 0.05, 128)
    q2, s2 = layer.norm(out)
    y = torch.empty(T, 200, device="cuda")
    cm.coli_fp8_matmul(q2, s2, head_q.cuda(), head_s.cuda(), y)
    want, bound = ref.matmul(q2.cpu(), s2.cpu(), head_q, head_s)
    assert (y.cpu().double() - want).abs().le(bound).all()
    assert cm.coli_moe_get_status() == (0, 0)


def test_empty_batches(cm):
    dims = cm.dims_for(256, 128, 4, 2, 1, group=128, code_bits=8)
    dev = {n: v.cuda() for n, v in _experts(4, 1, 256, 128, 30).items()}
    layer = cm.Fp8MoELayer(dims, dev)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, torch.empty(0, 4, device="cuda"), torch.empty_like(x), layer.workspace(0))
    cm.coli_fp8_matmul(torch.empty(0, 256, dtype=F8, device="cuda"), torch.empty(0, 2, device="cuda"), dev["gate_q"][0],
                       dev["gate_s"][0], torch.empty(0, 128, device="cuda"))
    assert cm.coli_moe_get_status() == (0, 0)


def test_expert_ffn_with_no_expert_at_all(cm):
    """Every id out of range and no shared expert: the residual comes back."""
    for T in (3, 90):
        dims = cm.dims_for(256, 128, 4, 2, 0, group=128, code_bits=8)
        t = _experts(4, 0, 256, 128, 40)
        g = torch.Generator().manual_seed(41)
        xq, xs = ref.block_quantise(torch.randn(T, 256, generator=g, dtype=torch.float64), 1)
        ids = torch.full((T, 2), -1, dtype=torch.int32)
        w = torch.full((T, 2), 0.5)
        r = torch.randn(T, 256, generator=g).to(torch.bfloat16)
        out = _ffn(cm, dims, t, xq, xs, ids, w, r)
        assert torch.equal(out.cpu(), r)
        assert cm.coli_moe_get_status()[1] == cm._lib.COLI_FLAG_BAD_ID


def test_expert_ffn_batch_boundaries(cm):
    """32 tokens and fewer take one form, 33 another; segments of 127, 128, 129 and
    256 tokens end on and beside a token block."""
    H, I = 256, 128
    for T, E, k, S in ((31, 3, 1, 1), (32, 3, 2, 0), (33, 3, 2, 1), (127, 1, 1, 0), (128, 1, 1, 1), (129, 1, 1, 0),
                       (256, 2, 2, 0), (257, 1, 1, 2)):
        dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
        t = _experts(E, S, H, I, T)
        g = torch.Generator().manual_seed(T)
        xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
        _, ids, w = _routed(T, E, k, T)
        out = _ffn(cm, dims, t, xq, xs, ids, w, None)
        want, bound = ref.expert_ffn(dims, t, xq, xs, ids, w, None)
        assert (out.cpu().double() - want).abs().le(bound).all(), (T, E, k, S)


# ------------------------------------------------- offsets past 32 bits --

def test_matmul_offsets_past_32_bits(cm):
    """2.3e9 results: rows from the start, the middle and the end."""
    M, N, K = 140_001, 16_392, 64
    g = torch.Generator(device="cuda").manual_seed(50)
    a = torch.randint(0, 120, (M, K), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    w = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    as_ = torch.rand(M, 1, device="cuda", generator=g)
    ws = torch.rand(-(-N // 128), 1, device="cuda", generator=g)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    cm.coli_fp8_matmul(a, as_, w, ws, out)
    rows = torch.tensor([0, 1, 65_535, 131_000, 131_071, 131_072, 140_000])
    want, bound = ref.matmul(a[rows.cuda()].cpu(), as_[rows.cuda()].cpu(), w.cpu(), ws.cpu())
    bound = bound + ref.UBF16 * (want.abs() + bound)
    assert (out[rows.cuda()].cpu().double() - want).abs().le(bound).all()
    assert cm.coli_moe_get_status() == (0, 0)


def test_norm_offsets_past_32_bits(cm):
    T, H = 70_003, 32_768
    g = torch.Generator(device="cuda").manual_seed(51)
    x = torch.randn(T, H, device="cuda", generator=g, dtype=torch.bfloat16)
    q = torch.empty(T, H, dtype=F8, device="cuda")
    sc = torch.empty(T, H // 128, device="cuda")
    n = torch.empty_like(x)
    cm.coli_add_rmsnorm_fp8(x, None, None, 1e-6, None, n, q, sc)
    rows = torch.tensor([0, 65_535, 65_536, 70_002]).cuda()
    v = x[rows].cpu().double()
    want = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert (n[rows].cpu().double() - want).abs().le((88 * U + ref.UBF16) * want.abs() + 1e-37).all()
    # half an e4m3 step of a normal value, half the smallest step (2^-10 scales) below
    deq = ref.decode(q[rows]) * ref.spread(sc[rows].cpu().double(), H, 1)
    assert (deq - want).abs().le(2.0 ** -4 * want.abs() * (1 + 200 * U) + 2.0 ** -10 * ref.spread(sc[rows].cpu().double(), H, 1)).all()


def test_expert_ffn_offsets_past_32_bits(cm):
    """2.2e9 values of y and of the gathered codes: tokens from both ends."""
    T, E, k, H, I = 44_001, 8, 8, 6_144, 128
    dims = cm.dims_for(H, I, E, k, 0, group=128, code_bits=8)
    t = _experts(E, 0, H, I, 52)
    dev = {m: v.cuda() for m, v in t.items()}
    g = torch.Generator(device="cuda").manual_seed(53)
    xq = torch.randint(0, 120, (T, H), dtype=torch.uint8, device="cuda", generator=g)
    xq = (xq + 128 * torch.randint(0, 2, (T, H), dtype=torch.uint8, device="cuda", generator=g)).view(F8)
    xs = 0.01 * torch.rand(T, H // 128, device="cuda", generator=g)
    top, ids = torch.topk(torch.randn(T, E, device="cuda", generator=g), k, dim=1)
    ids, w = ids.to(torch.int32), torch.softmax(top, 1)
    arrays = ref.union(ids, E)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(cm.coli_moe_fp8_workspace_bytes(dims, T), dtype=torch.uint8, device="cuda")
    cm.coli_moe_expert_ffn_fp8(dims, cm.fp8_weights(**dev), xq, xs, ids, w, *arrays, None, out, ws)
    rows = torch.tensor([0, 1, 22_000, 43_999, 44_000]).cuda()
    want, bound = ref.expert_ffn(dims, t, xq[rows].cpu(), xs[rows].cpu(), ids[rows].cpu(), w[rows].cpu(), None)
    err = (out[rows].cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())
    assert cm.coli_moe_get_status() == (0, 0)


def test_norm_codes_are_the_nearest(cm):
    """Away from the ends of fp32 a code is the nearest one to the exact ratio 448 s g
    / max|s g|: two fp32 roundings before the code's own (the quotient 448 / max, the
    product), half a step 2^-24 each, (1 + 2^-24)^2 - 1 < 2.01 * 2^-24: only a ratio
    within that of a border may land on its other side."""
    g = torch.Generator().manual_seed(70)
    x = (3 * torch.randn(600, 6144, generator=g)).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(6144, generator=g)).to(torch.bfloat16)
    for weight in (w, None):
        q = torch.empty(600, 6144, dtype=F8, device="cuda")
        sc = torch.empty(600, 48, device="cuda")
        cm.coli_add_rmsnorm_fp8(x.cuda(), None, None if weight is None else weight.cuda(), 1e-6, None, None, q, sc)
        y = x.double() * (1 if weight is None else weight.double())
        v = 448 * y / ref.spread(y.abs().view(600, -1, 128).amax(-1), 6144, 1)
        got = ref.decode(q)
        lo, hi = ref.e4m3_round(v * (1 - 2.01 * U)), ref.e4m3_round(v * (1 + 2.01 * U))
        assert ((got == lo) | (got == hi)).all()


def test_norm_of_extreme_weights(cm):
    """Weights whose product with the row leaves fp32's exact range: the codes then
    come from n itself."""
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(71)).to(torch.bfloat16)
    for w in (1e37, 1e-30):
        _norm_check(cm, x, None, torch.full((256,), w).to(torch.bfloat16))
