"""Tall and narrow products whose K is split over CTAs and summed by a second kernel: outputs of a few
columns, whole and odd, beside guard bytes, in both formats."""
import pytest
import torch

import nvfp4_block_scaled_14_b200 as nv
from nvfp4_block_scaled_14_b200 import _lib as L
from test_mxfp4 import check_product, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


SHAPES = [(4096, 8, 1024), (8192, 16, 1024), (3001, 30, 512), (130, 1, 2048), (1000, 3, 544),
          (2050, 129, 1056), (400, 1998, 512), (200, 264, 8192), (130, 30, 29984),
          (777, 1001, 2080)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_mxfp4(M, N, K, out):
    assert L.load().nvfp4_workspace_bytes(L.NVFP4_OP_LINEAR, M, N, K) > 0  # K is split
    a, va = operand(M, K, 1)
    w, vw = operand(N, K, 2)
    pad = 64
    buf = torch.full((M * N + 2 * pad,), -77.0, dtype=out, device="cuda")
    y = buf[pad:-pad].view(M, N)
    check_product(nv.linear_mxfp4(a, w, out, out=y), va, vw, f"{M}x{N}x{K}")
    assert (buf[:pad] == -77.0).all() and (buf[-pad:] == -77.0).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nvfp4(M, N, K):
    """Both operands +-1 and +-2 with unit scales: every sum is a small integer, exact in fp32."""
    g = torch.Generator(device="cuda").manual_seed(M + N)

    def ones(rows):
        # codes of +-1 and +-2, two a byte; scales of 1 in every atom, padding included
        n = torch.tensor([2, 4, 10, 12], device="cuda")[
            torch.randint(0, 4, (rows, K), device="cuda", generator=g)]
        v = torch.where(n >= 8, -1.0, 1.0) * torch.where(n & 7 == 2, 1.0, 2.0)
        codes = (n[:, 0::2] | n[:, 1::2] << 4).to(torch.uint8).contiguous()
        swz = torch.full((L.load().nvfp4_scales_bytes(rows, K, 1),), 0x38, dtype=torch.uint8,
                         device="cuda")
        return nv.NVFP4Tensor(codes, swz, None, torch.ones(1, device="cuda"), rows, K), v.double()
    (a, va), (w, vw) = ones(M), ones(N)
    ref = va @ vw.T
    assert torch.equal(nv.linear(a, w, torch.float32).double(), ref)
    assert torch.equal(nv.linear(a, w), ref.bfloat16())
