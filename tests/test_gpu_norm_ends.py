"""The norm with 8-bit rows at the ends of fp32: rows whose squares vanish or overflow,
next to no eps, rows of zeros without any."""
import pytest
import torch

from tests import _fp8 as ref
from tests._gpu import needs_gpu
from tests.test_gpu_fp8 import _norm_check

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    m.coli_moe_get_status()
    return m


def _rows(H, seed):
    """Rows of many magnitudes in one call; every value is a bf16 number, the smallest
    of them subnormal ones of a few bits."""
    g = torch.Generator().manual_seed(seed)
    scales = [1.0, 1e-18, 1e-20, 1e-24, 1e-30, 1e-37, 1e-39, 3e-41, 1e18, 1e20, 1e30, 1e37]
    x = torch.randn(len(scales), H, generator=g).clamp(-3, 3)
    return (x * torch.tensor(scales, dtype=torch.float64)[:, None]).to(torch.bfloat16)


@pytest.mark.parametrize("H", [128, 1024, 2176, 6144, 8192, 16384, 32768])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -120, 1e-6])
def test_rows_of_every_magnitude(cm, H, eps):
    """_norm_check's bounds: a power of two more changes no rounding."""
    x = _rows(H, H)
    w = (1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    for weight in (None, w):
        _norm_check(cm, x, None, weight, eps=eps)
    assert cm.coli_moe_get_status() == (0, 0)


def test_with_a_residual_and_in_place(cm):
    x, r = _rows(640, 3), _rows(640, 4)
    for kw in (dict(), dict(in_place="x"), dict(in_place="r", want_norm=False)):
        _norm_check(cm, x, r, None, eps=0.0, **kw)
    assert cm.coli_moe_get_status() == (0, 0)


def test_a_loud_value_among_small_ones(cm):
    """The row's power of two comes from its largest value; the others keep their place."""
    x = _rows(384, 5)
    x[:, 7] = x.float().abs().amax(1).mul(100).clamp_max(3e38).to(torch.bfloat16)
    _norm_check(cm, x, None, None, eps=0.0)
    assert cm.coli_moe_get_status() == (0, 0)


@pytest.mark.parametrize("H", [256, 6144, 16384])
def test_zeros_stay_zeros_without_eps(cm, H):
    """Padding rows between others, their outputs prefilled with something else."""
    x = torch.zeros(4, H, dtype=torch.bfloat16)
    x[1] = torch.randn(H, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    x[3, ::2] = -0.0
    q = torch.full((4, H), 0x55, dtype=torch.uint8, device="cuda")
    sc, n = torch.full((4, H // 128), 7.0, device="cuda"), torch.full((4, H), 7.0, dtype=torch.bfloat16, device="cuda")
    cm.coli_add_rmsnorm_fp8(x.cuda(), None, None, 0.0, None, n, q, sc)
    for t in (0, 2, 3):
        assert (q[t] & 0x7F == 0).all() and (n[t] == 0).all() and (sc[t] == 2.0 ** -126).all()
    want = x[1].double() / torch.sqrt((x[1].double() ** 2).mean())
    assert (n[1].cpu().double() - want).abs().le((88 * ref.U32 + ref.UBF16) * want.abs()).all()
    assert cm.coli_moe_get_status() == (0, 0)


def test_infinities_and_nan_are_flagged(cm):
    """An infinity leaves NaN in its block and zeros elsewhere, NaN its whole row; a sum
    with the residual that overflows is an infinity; other rows are untouched."""
    x = torch.ones(5, 512, dtype=torch.bfloat16)
    x[1, 130] = float("inf")
    x[2, 9] = float("nan")
    x[3, 300] = 3e38
    r = torch.zeros(5, 512, dtype=torch.bfloat16)
    r[3, 300] = 3e38
    for row in (1, 2, 3):
        cm.coli_moe_get_status()
        q, sc = torch.empty(1, 512, dtype=torch.uint8, device="cuda"), torch.empty(1, 4, device="cuda")
        cm.coli_add_rmsnorm_fp8(x[row:row + 1].cuda(), r[row:row + 1].cuda(), None, 1e-6, None, None, q, sc)
        assert cm.coli_moe_get_status()[1] == cm._lib.COLI_FLAG_NONFINITE, row
        q, bad = q.cpu()[0], torch.isnan(sc.cpu()[0])
        want = {1: [False, True, False, False], 2: [True] * 4, 3: [False, False, True, False]}[row]
        assert bad.tolist() == want
        for b in range(4):
            assert (q[128 * b:128 * b + 128] == (0x7F if want[b] else 0)).all()
    q, sc = torch.empty(5, 512, dtype=torch.uint8, device="cuda"), torch.empty(5, 4, device="cuda")
    cm.coli_add_rmsnorm_fp8(x.cuda(), r.cuda(), None, 1e-6, None, None, q, sc)
    assert (q[0] == q[4]).all() and (q[0] == 0x7E).all() and torch.isfinite(sc[[0, 4]]).all()
    cm.coli_moe_get_status()
