"""What the e4m3 expert set and its holder refuse.  CPU only: the tensors say that
they are in device memory, and no call reaches the library."""
import pytest
import torch


@pytest.fixture(scope="module")
def cm():
    from int4_routed_expert_renorm_b200.build import build
    build()
    import int4_routed_expert_renorm_b200 as m
    return m


class Dev:
    """A tensor of this shape and type that says it is on GPU `gpu`."""

    def __init__(self, shape, dtype, gpu=0, address=0x10000):
        self.shape, self.dtype, self.gpu, self.address = torch.Size(shape), dtype, gpu, address
        self.is_cuda, self.device = True, torch.device("cuda", gpu)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return self.address

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


SHAPES = {"gate_q": (5, 128, 256), "up_q": (5, 128, 256), "down_q": (5, 256, 128),
          "gate_s": (5, 1, 2), "up_s": (5, 1, 2), "down_s": (5, 2, 1)}


def _set(codes=torch.float8_e4m3fn, scales=torch.float32, **other):
    t = {n: Dev(s, codes if n[-1] == "q" else scales) for n, s in SHAPES.items()}
    for n, kw in other.items():
        t[n] = Dev(**{**dict(shape=SHAPES[n], dtype=t[n].dtype), **kw})
    return t


@pytest.mark.parametrize("codes", [torch.float8_e4m3fn, torch.uint8, torch.int8])
def test_weights_accept_codes_and_their_bytes(cm, codes):
    w = cm.fp8_weights(**_set(codes))
    assert (w.gate_q, w.down_s) == (0x10000, 0x10000)


@pytest.mark.parametrize("name", ["gate_q", "up_q", "down_q"])
@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.bool,
                                   torch.bfloat16])
def test_weights_refuse_codes_of_another_format(cm, name, dtype):
    with pytest.raises(ValueError, match=f"{name}.*float8_e4m3fn"):
        cm.fp8_weights(**_set(**{name: dict(dtype=dtype)}))


@pytest.mark.parametrize("name", ["gate_s", "up_s", "down_s"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.uint32, torch.float64, torch.bfloat16])
def test_weights_refuse_scales_of_another_type(cm, name, dtype):
    with pytest.raises(ValueError, match=f"{name}.*float32"):
        cm.fp8_weights(**_set(**{name: dict(dtype=dtype)}))


@pytest.mark.parametrize("name", list(SHAPES)[1:])
def test_weights_refuse_tensors_of_two_devices(cm, name):
    with pytest.raises(ValueError, match=f"{name}.*cuda:1"):
        cm.fp8_weights(**_set(**{name: dict(gpu=1)}))


def _call(cm, dims, weights, T=3):
    H, P = dims.hidden, T * dims.top_k
    U = min(dims.n_experts, P)
    i32 = lambda *s: Dev(s, torch.int32)  # noqa: E731
    ws = Dev((1 << 20,), torch.uint8)
    ws.nbytes = 1 << 20
    cm.coli_moe_expert_ffn_fp8(dims, weights, Dev((T, H), torch.uint8), Dev((T, H // 128), torch.float32),
                               i32(T, dims.top_k), Dev((T, dims.top_k), torch.float32), i32(U), i32(1), i32(U + 1), i32(P),
                               i32(P), None, Dev((T, H), torch.bfloat16), ws, 0)


@pytest.fixture
def no_launch(cm, monkeypatch):
    """The C entry counts its calls instead; the current device is GPU 0."""
    class Lib:
        calls = 0

        def coli_moe_expert_ffn_fp8(self, *a):
            Lib.calls += 1
            return 0

    monkeypatch.setattr(cm._lib, "_lib", Lib())
    monkeypatch.setattr(cm._lib, "_current_device", lambda: 0)
    return Lib


@pytest.mark.parametrize("E,S,I,H", [(5, 1, 128, 256), (3, 1, 128, 256), (4, 1, 256, 256), (4, 1, 128, 384), (4, 2, 128, 256)])
def test_call_refuses_weights_of_other_dims(cm, no_launch, E, S, I, H):
    """More experts or longer rows than the set has would be read past its end."""
    with pytest.raises(ValueError, match="weights: 5 experts of 128 x 256"):
        _call(cm, cm.dims_for(H, I, E, 2, S, group=128, code_bits=8), cm.fp8_weights(**_set()))
    assert no_launch.calls == 0


def test_call_refuses_weights_on_another_device(cm, no_launch):
    t = {n: Dev(s, torch.uint8 if n[-1] == "q" else torch.float32, gpu=1) for n, s in SHAPES.items()}
    dims = cm.dims_for(256, 128, 4, 2, 1, group=128, code_bits=8)
    with pytest.raises(ValueError, match="weights: tensors on cuda:1, but the call runs on cuda:0"):
        _call(cm, dims, cm.fp8_weights(**t))
    assert no_launch.calls == 0
    _call(cm, dims, cm.fp8_weights(**_set()))
    _call(cm, cm.dims_for(256, 128, 5, 2, 0, group=128, code_bits=8), cm.fp8_weights(**_set()))   # the same 5 experts
    _call(cm, dims, cm.coli_moe_weights_fp8(*[0x10000] * 6))       # by hand: the caller answers for it
    assert no_launch.calls == 3


def test_layer_checks_its_norm_weight_when_it_is_built(cm):
    dims = cm.dims_for(256, 128, 4, 2, 1, group=128, code_bits=8)
    strided = Dev((256,), torch.bfloat16)
    strided.is_contiguous = lambda: False
    for bad in (Dev((128,), torch.bfloat16), Dev((256,), torch.float32), Dev((256,), torch.float16),
                Dev((256,), torch.bfloat16, gpu=1), torch.ones(256, dtype=torch.bfloat16), strided):
        with pytest.raises(ValueError, match="norm_weight"):
            cm.Fp8MoELayer(dims, _set(), bad)
    for good in (None, Dev((256,), torch.bfloat16), Dev((256,), torch.int16)):
        assert cm.Fp8MoELayer(dims, _set(), good).norm_weight is good


def test_binding_without_the_quick_device_and_stream_lookups(cm, monkeypatch):
    """On a torch without them the public forms answer: the call reaches the library
    with the current stream's handle."""
    import importlib.util
    from types import SimpleNamespace
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=0x70 + device))
    spec = importlib.util.spec_from_file_location("int4_routed_expert_renorm_b200._lib_other", cm._lib.__file__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    seen = []
    other._lib = SimpleNamespace(coli_fp8_matmul=lambda *a: seen.append(a) or 0)
    a, w = Dev((3, 256), torch.uint8), Dev((128, 256), torch.uint8)
    other.coli_fp8_matmul(a, Dev((3, 2), torch.float32), w, Dev((1, 2), torch.float32), Dev((3, 128), torch.float32))
    assert len(seen) == 1 and seen[0][-1] == 0x70
    with pytest.raises(ValueError, match="current device is cuda:0"):
        other.coli_fp8_matmul(Dev((3, 256), torch.uint8, gpu=1), Dev((3, 2), torch.float32), w, Dev((1, 2), torch.float32),
                              Dev((3, 128), torch.float32))
