"""Few-token products over numbers of tiles at which the split of k changes:
as many clusters as the GPU holds at once, and one more or less."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

from _ops_ref import check_product
from test_gpu_fp8_blocks import operands, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tiles", [35, 36, 37, 38, 39, 73, 74, 75, 76, 77, 151, 152, 153])
@pytest.mark.parametrize("T,dtype", [(1, torch.float32), (20, torch.bfloat16), (64, torch.float8_e4m3fn), (70, torch.float32)])
def test_product_where_the_split_changes(tiles, T, dtype):
    x, xs, w, ws = operands(T, 1, 128 * tiles - 3, 1040, tiles)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, scales = product(x, xs, w, ws, dtype, status=status)
    check_product(out, x, xs, w, ws, scales)
    again, scales2 = product(x, xs, w, ws, dtype)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8)) and (scales is None or torch.equal(scales, scales2))
    assert B.read_device_status(status)[0] == B.OK
