"""The holders' own arrays belong to the stream that their calls run on.  CPU only:
the library's calls and the allocator's current stream are fakes."""
import contextlib

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def cm():
    from int4_routed_expert_renorm_b200.build import build
    build()
    import int4_routed_expert_renorm_b200 as m
    return m


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def made(monkeypatch):
    """address -> stream that was current when a tensor was made (None: the default one)."""
    now, where, keep = [None], {}, []

    @contextlib.contextmanager
    def scope(stream):
        now.append(stream)
        yield
        now.pop()

    def recorded(make):
        def f(*a, **kw):
            t = make(*a, **kw)
            where[t.data_ptr()] = now[-1]
            keep.append(t)           # no address is handed out twice
            return t
        return f

    monkeypatch.setattr(torch.cuda, "stream", scope)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    for name in ("empty", "empty_like", "from_numpy"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "contiguous", recorded(torch.Tensor.contiguous))
    return where


def _calls(monkeypatch, module, names):
    seen = []
    for name in names:
        monkeypatch.setattr(module, name, lambda *a, _n=name, **kw: seen.append((_n, a)))
    return seen


@pytest.mark.parametrize("stream", [None, FakeStream(0x70), 0x70])
def test_fp8_layer(cm, monkeypatch, made, stream):
    """norm, experts and forward: what the kernels on `stream` read and write, and the
    caller did not bring, was made under that stream."""
    layer = object.__new__(cm.Fp8MoELayer)
    layer.dims = cm.dims_for(256, 128, 8, 2, 1, group=128, code_bits=8)
    layer.weights, layer.norm_weight, layer.eps = None, torch.zeros(256, dtype=torch.bfloat16), 1e-6
    seen = _calls(monkeypatch, cm.fp8, ("coli_add_rmsnorm_fp8", "coli_moe_route", "coli_moe_union",
                                        "coli_moe_expert_ffn_fp8"))
    x, r = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, 256, dtype=torch.bfloat16)
    out, logits, ws = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, 8), torch.zeros(16, dtype=torch.uint8)
    own = {t.data_ptr() for t in (x, r, out, logits, ws, layer.norm_weight)}
    made.clear()
    ids, w = layer.forward(x, logits, out, ws, residual=r, stream=stream)
    q, s = layer.norm(x, stream=stream)
    layer.experts(q, s, ids, w, out, ws, stream=stream)
    assert [n for n, _ in seen] == ["coli_add_rmsnorm_fp8", "coli_moe_route", "coli_moe_union", "coli_moe_expert_ffn_fp8",
                                    "coli_add_rmsnorm_fp8", "coli_moe_union", "coli_moe_expert_ffn_fp8"]
    used = 0
    for name, args in seen:
        assert args[-1] is stream, name
        for t in args:
            if isinstance(t, torch.Tensor) and t.data_ptr() not in own:
                on = made[t.data_ptr()]
                assert (on is None) if stream is None else (on is not None and on.cuda_stream == 0x70), (name, t.shape)
                used += 1
    assert used >= 2 * (2 + 2 + 5 + 5)


@pytest.mark.parametrize("stream", [None, FakeStream(0x70), 0x70])
def test_tier_warm_start(cm, monkeypatch, made, stream):
    """The profile's words, the hottest experts' ids and a dense copy of strided ids
    are made and copied on the stream that places them."""
    dims = cm.dims_for(256, 256, 8, 2, 0)
    tl = object.__new__(cm.TieredLayer)
    tl.dims, tl.n_slots, tl.weights, tl.tier = dims, 3, None, None
    tl.state = torch.zeros(4 * (8 + 3 + 8 + 64), dtype=torch.uint8)
    copies = []
    copy = torch.Tensor.copy_
    monkeypatch.setattr(torch.Tensor, "copy_", lambda a, b: (copies.append(torch.empty(1)), copy(a, b))[1])
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: None)
    seen = _calls(monkeypatch, cm.tier, ("coli_moe_tier_prefetch",))
    tl.warm_from_usage(np.array([5, 0, 9, 1, 7, 0, 0, 2]), stream)
    tl.prefetch(torch.arange(6, dtype=torch.int32)[::2], stream)
    assert [a[3].tolist() for _, a in seen] == [[2, 4, 0], [0, 2, 4]] and len(copies) == 1
    for t in copies + [a[3] for _, a in seen]:
        on = made[t.data_ptr()]
        assert (on is None) if stream is None else (on is not None and on.cuda_stream == 0x70)
    assert all(a[-1] is stream for _, a in seen)
    assert tl.state.view(torch.int32)[11:19].tolist() == [5, 0, 9, 1, 7, 0, 0, 2]
