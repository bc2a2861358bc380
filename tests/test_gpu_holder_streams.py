"""Holders called on another stream than the current one, which goes on allocating
and writing blocks of the sizes that the holder's own arrays have."""
import pytest
import torch

from tests import _fp8 as ref
from tests._gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    return m


def _fp8_layer(cm, dims, seed):
    g = torch.Generator().manual_seed(seed)
    t = {}
    n, H, I = dims.n_experts + dims.n_shared, dims.hidden, dims.inter
    for name, R, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        q, s = ref.block_quantise(torch.randn(n, R, K, generator=g, dtype=torch.float64) / K ** 0.5, 128)
        t[name + "_q"], t[name + "_s"] = q.cuda(), s.cuda()
    return cm.Fp8MoELayer(dims, t, (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda())


@pytest.mark.parametrize("T", [7, 90])           # gathered copies; pair order
@pytest.mark.parametrize("handle", ["stream", "number", "default"])
def test_fp8_layer_on_another_stream(cm, T, handle):
    """The other stream is held up by 20 ms or so, so that its kernels run behind the
    current stream's writes.  Every array of the call keeps its contents: the bits of
    the call on the current stream."""
    E, k, S, H, I = 12, 3, 1, 384, 256
    layer = _fp8_layer(cm, cm.dims_for(H, I, E, k, S, group=128, code_bits=8), T)
    g = torch.Generator().manual_seed(T + 1)
    x, r = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    logits = torch.randn(T, E, generator=g).cuda()
    ws = layer.workspace(T)
    want = torch.empty_like(x)
    want_ids, want_w = layer.forward(x, logits, want, ws, residual=r)
    want_q, want_s = layer.norm(x, r)
    out = torch.zeros_like(x)
    side = torch.cuda.default_stream() if handle == "default" else torch.cuda.Stream()
    current = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        arg = side if handle == "stream" else side.cuda_stream
        ids, w = layer.forward(x, logits, out, ws, residual=r, stream=arg)
        q, s = layer.norm(x, r, stream=arg)
        sizes = [x.nbytes, T * H, T * H // 32, 4 * T * k, 4 * min(E, T * k), 4 * (min(E, T * k) + 1), 4]
        spoil = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        assert len(spoil) == 28
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(ids, want_ids) and torch.equal(w, want_w)
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    assert cm.coli_moe_get_status() == (0, 0)


def test_tier_warm_start_on_another_stream(cm):
    """The usage profile and the placement follow each other on the given stream, held
    up here while the current stream writes blocks of their sizes."""
    import numpy as np
    import synth
    import synth.gpu as sg
    E, k, C = 32, 2, 6
    shape = synth.LayerShape("tier_side", 512, 256, E, k, 1, 2)
    dims = cm.dims_for(512, 256, E, k, 1)
    tl = cm.TieredLayer(dims, sg.expert_tensors(shape), C)
    profile = np.zeros(E, np.int64)
    profile[[3, 9, 10, 21, 30, 31, 7]] = [50, 40, 40, 30, 20, 20, 20]
    side = torch.cuda.Stream()
    ids = torch.tensor([5, 0, 6, 0], dtype=torch.int32, device="cuda")[::2]
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        tl.reset()
        tl.warm_from_usage(profile, stream)
        spoil = [torch.full((n,), 1, dtype=torch.int32, device="cuda") for n in (C, E) for _ in range(4)]
        st = tl.state_arrays()
        assert sorted(st["owner"].tolist()) == [3, 7, 9, 10, 21, 30] and len(spoil) == 8
        assert np.array_equal(st["usage"], profile.astype(np.uint32))
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        tl.prefetch(ids, stream)                # strided: the holder makes a dense copy
        spoil = [torch.full((2,), 1, dtype=torch.int32, device="cuda") for _ in range(4)]
        owner = tl.state_arrays()["owner"].tolist()
        assert 5 in owner and 6 in owner and 1 not in owner
    assert cm.coli_moe_get_status() == (0, 0)


@pytest.mark.parametrize("fork", [False, True])
def test_fp8_layer_in_a_graph(cm, fork):
    """forward captured, on the capturing stream or on one that forks from it and joins
    again, and replayed with other inputs while eager calls run in between."""
    T, E, k, S, H, I = 40, 12, 3, 1, 384, 256
    layer = _fp8_layer(cm, cm.dims_for(H, I, E, k, S, group=128, code_bits=8), 5)
    g = torch.Generator().manual_seed(6)
    ins = [[torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
           + [torch.randn(T, E, generator=g).cuda()] for _ in range(3)]
    ws, ws2 = layer.workspace(T), layer.workspace(T)

    def eager(x, r, logits):
        out = torch.empty_like(x)
        ids, w = layer.forward(x, logits, out, ws, residual=r)
        return out, ids, w

    want = [eager(*i) for i in ins]
    x, r, logits = (t.clone() for t in ins[0])
    out, side = torch.zeros_like(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if fork:
            side.wait_stream(torch.cuda.current_stream())
            ids, w = layer.forward(x, logits, out, ws2, residual=r, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        else:
            ids, w = layer.forward(x, logits, out, ws2, residual=r)
    for i, (o, oi, ow) in zip(ins, want):
        for dst, src in zip((x, r, logits), i):
            dst.copy_(src)
        graph.replay()
        again = eager(*i)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(ids, oi) and torch.equal(w, ow)
        assert torch.equal(again[0], o)
    assert cm.coli_moe_get_status() == (0, 0)
