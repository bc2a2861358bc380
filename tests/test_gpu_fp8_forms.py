"""The 8-bit product's kernels in their lasting form: CTAs that take several tiles one
after the other, each of several K blocks, so that barriers, stages, scales and the
tile's totals are carried from one tile to the next.  Sizes are chosen by the tiles
that they make on a GPU of 148 SMs; the results are checked on any."""
import pytest
import torch

from tests import _fp8 as ref
from tests._gpu import needs_gpu
from tests.test_gpu_fp8 import _experts, _ffn, _routed

pytestmark = [pytest.mark.gpu, needs_gpu]
F8 = ref.F8


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    m.coli_moe_get_status()
    return m


def _codes(g, *shape):
    """Random finite codes of both signs."""
    mag = torch.randint(0, 0x7F, shape, dtype=torch.uint8, generator=g)
    return (mag + 128 * torch.randint(0, 2, shape, dtype=torch.uint8, generator=g)).view(F8)


def _check_matmul(cm, M, N, K, f32, seed):
    g = torch.Generator().manual_seed(seed)
    nk, nrb = -(-K // 128), -(-N // 128)
    aq, wq = _codes(g, M, K), _codes(g, N, K)
    as_, ws = torch.rand(M, nk, generator=g) + 0.01, torch.rand(nrb, nk, generator=g) + 0.01
    pad = 64
    buf = torch.full((M * N + pad,), 7, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    out = buf[:M * N].view(M, N)
    cm.coli_fp8_matmul(aq.cuda(), as_.cuda(), wq.cuda(), ws.cuda(), out)
    torch.cuda.synchronize()
    assert (buf[M * N:] == 7).all()
    want, bound = ref.matmul(aq, as_, wq, ws)
    if not f32:
        bound = bound + ref.UBF16 * (want.abs() + bound)
    err = (out.cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())
    assert cm.coli_moe_get_status() == (0, 0)


@pytest.mark.parametrize("M,N,K", [
    (1, 40001, 400),       # up to 32 rows, two weight blocks a tile: 157 tiles, the last one of a single block
    (17, 40008, 272),      # 157 tiles, 3 K blocks
    (32, 76032, 656),      # 297 tiles, three for one CTA; 6 K blocks: the scales' groups of four end in the middle
    (32, 57088, 1168),     # 223 tiles; 10 K blocks, more than the stages
    (5, 20001, 400),       # one weight block a tile: 157 tiles
    (32, 32768, 784),      # 256 tiles of one block
])
@pytest.mark.parametrize("f32", [True, False])
def test_few_rows(cm, M, N, K, f32):
    _check_matmul(cm, M, N, K, f32, M + N + K)


@pytest.mark.parametrize("M,N,K", [
    (2048, 4100, 1040),    # two weight blocks a tile: 272 tiles of 9 K blocks
    (1100, 8200, 528),     # 297 tiles of 5, token blocks of 122 and 123 rows
    (700, 15001, 144),     # 354 tiles of 2
    (1024, 2500, 656),     # one weight block a tile: 160 tiles of 6
    (290, 9473, 400),      # 225 tiles of 4, odd rows
])
@pytest.mark.parametrize("f32", [True, False])
def test_many_rows(cm, M, N, K, f32):
    _check_matmul(cm, M, N, K, f32, M + N + K)


@pytest.mark.parametrize("T,E,k,S,H,I", [
    (32, 64, 8, 0, 640, 1024),     # 512 gate/up tiles with gathered rows, 5 K blocks; 320 down tiles, 8
    (20, 40, 6, 2, 1152, 640),     # 200 gate/up tiles, 9 K blocks; 360 down tiles, 5
    (700, 10, 2, 0, 2944, 1408),   # 187 gate/up tiles, 23 K blocks; 204 down tiles, 11
    (300, 24, 3, 1, 1408, 896),    # segments of about 37 tokens, a shared one of 300: 189 tiles, 11; 162, 7
])
def test_expert_ffn(cm, T, E, k, S, H, I):
    dims = cm.dims_for(H, I, E, k, S, group=128, code_bits=8)
    t = _experts(E, S, H, I, T)
    g = torch.Generator().manual_seed(T + 1)
    xq, xs = ref.block_quantise(torch.randn(T, H, generator=g, dtype=torch.float64), 1)
    _, ids, w = _routed(T, E, k, T + 2)
    residual = torch.randn(T, H, generator=g).to(torch.bfloat16)
    out = _ffn(cm, dims, t, xq, xs, ids, w, residual)
    want, bound = ref.expert_ffn(dims, t, xq, xs, ids, w, residual)
    err = (out.cpu().double() - want).abs()
    assert err.le(bound).all(), float((err / bound).max())
    assert cm.coli_moe_get_status() == (0, 0)


def test_rows_of_batches_of_other_sizes(cm):
    """The same row in batches of 1 to 1500: the bits repeat call by call; between
    batches K may be split over other numbers of CTAs, and both are within the sums'
    bound of the exact product."""
    g = torch.Generator().manual_seed(9)
    N, K = 1001, 1552
    aq, wq = _codes(g, 1500, K), _codes(g, N, K)
    as_, ws = torch.rand(1500, 13, generator=g), torch.rand(8, 13, generator=g)
    A, SA, W, SW = aq.cuda(), as_.cuda(), wq.cuda(), ws.cuda()
    want, bound = ref.matmul(aq[:1], as_[:1], wq, ws)
    for M in (1, 2, 31, 32, 33, 127, 128, 129, 300, 700, 1500):
        outs = [torch.empty(M, N, device="cuda") for _ in range(2)]
        for out in outs:
            cm.coli_fp8_matmul(A[:M].contiguous(), SA[:M].contiguous(), W, SW, out)
        assert torch.equal(*outs), M
        assert (outs[0][:1].cpu().double() - want).abs().le(bound).all(), M
    assert cm.coli_moe_get_status() == (0, 0)
