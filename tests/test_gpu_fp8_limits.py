"""The FP8 block quantiser and product at the ends of their ranges: rows whose
lengths are near 2^31."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [2 ** 31 - 16, 2 ** 31 - 112, 2 ** 31 - 128, 2 ** 31 - 144])
def test_product_of_the_longest_rows(k):
    """k + 127 passes 2^31.  A few codes that are not zero, one in the last
    block: every product and sum is exact in fp32."""
    blocks = -(-k // 128)
    at = torch.tensor([0, 5, 128 * 77 + 3, k // 2, 128 * (blocks - 1), k - 1], device="cuda")
    x, w = torch.zeros((1, k), dtype=torch.uint8, device="cuda"), torch.zeros((1, k), dtype=torch.uint8, device="cuda")
    values = torch.tensor([1.0, 2.0, -4.0, 8.0, 0.5, 3.0], device="cuda")
    x[0, at] = values.to(torch.float8_e4m3fn).view(torch.uint8)
    w[0, at] = torch.full_like(values, 1.5).to(torch.float8_e4m3fn).view(torch.uint8)
    xs, ws = torch.full((1, blocks), 2.0, device="cuda"), torch.full((1, blocks), 4.0, device="cuda")
    xs[0, -1] = 16.0
    out, status = torch.full((1, 1), -1.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.fp8_block_matmul(x, xs, B.Fp8Weights(w, ws), out, status=status)
    scale = torch.where(at // 128 == blocks - 1, 64.0, 8.0)
    assert float(out) == float((values * 1.5 * scale).sum())
    assert B.read_device_status(status)[0] == B.OK


def pattern(dtype):
    """Three blocks of 128 values, each with a scale of its own."""
    g = torch.Generator().manual_seed(2)
    return (torch.randn((3, 128), generator=g) * torch.tensor([[1.0], [30.0], [0.02]])).to(dtype).cuda()


def quantise_long_rows(rows, cols, block_rows, dtype):
    """Rows that repeat three blocks, between large values that belong to no
    row; every code, scale and byte around them is checked."""
    pad = 64                                                        # behind each row, and ahead of the first
    step = (cols + pad + 15) // 16 * 16
    guard = float(torch.finfo(dtype).max)
    x = torch.full((pad + rows * step,), guard, dtype=dtype, device="cuda")[pad:].view(rows, step)
    p = pattern(dtype)
    whole = cols // 384
    for r in range(rows):
        x[r, :whole * 384].view(whole, 384).copy_(p.flatten().expand(whole, 384))
        x[r, whole * 384:cols] = p.flatten()[:cols - whole * 384]
    codes = torch.full((rows, step), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((1 if block_rows == 128 else rows, -(-cols // 128) + 2), -3.0, device="cuda")
    B.fp8_block_quant(x[:, :cols], codes[:, :cols], scales[:, :-2], block_rows=block_rows)
    del x
    # the last block may be partly filled
    last = cols % 128 or 128
    s = p.float().abs().amax(1) / torch.full((3,), 448.0, device="cuda")
    want = (p.float() / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten()
    blocks = -(-cols // 128)
    edge = p[(blocks - 1) % 3, :last].float()
    edge_s = edge.abs().amax() / torch.full((), 448.0, device="cuda")
    for r in range(rows):
        full = (cols - last) // 384
        assert bool((codes[r, :full * 384].view(full, 384) == want).all())
        assert torch.equal(codes[r, full * 384:cols - last], want[:cols - last - full * 384])
        assert torch.equal(codes[r, cols - last:cols], (edge / edge_s).to(torch.float8_e4m3fn).view(torch.uint8))
        assert bool((codes[r, cols:] == 0x55).all())
    for got in scales:
        assert bool((got[:blocks - 1] == s.repeat(-(-blocks // 3))[:blocks - 1]).all())
        assert float(got[blocks - 1]) == float(edge_s) and bool((got[blocks:] == -3).all())


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31 - 8])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_of_the_longest_rows(cols, block_rows, dtype):
    """The last lanes' columns end within a chunk of 2^31."""
    quantise_long_rows(1, cols, block_rows, dtype)


def test_quant_of_several_of_the_longest_rows():
    """Enough rows for the kernel of many blocks."""
    quantise_long_rows(7, 2 ** 31 - 8, 1, torch.bfloat16)
