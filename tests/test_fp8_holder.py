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
