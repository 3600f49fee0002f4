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
