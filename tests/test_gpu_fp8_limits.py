"""The FP8 block quantiser and product at the ends of their ranges: rows whose
lengths are near 2^31."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    """These buffers are tens of GB: none stay reserved for later tests."""
    yield
    torch.cuda.empty_cache()


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


def product_against_doubles(T, G, N, K, dtype, seed):
    """Operands and 64-bit sums on the GPU, in slices of tokens; k is one
    partly filled block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: (torch.randn(s, generator=g, device="cuda", dtype=torch.float32) * 4).to(torch.float8_e4m3fn)  # noqa: E731
    x, w = rand(T, G, K), rand(G, N, K)
    xs = torch.rand((T, G, 1), generator=g, device="cuda") + 0.5
    ws = torch.rand((G, -(-N // 128), 1), generator=g, device="cuda") + 0.5
    quant = dtype == torch.float8_e4m3fn
    out = torch.full((T, G, N), 18.0, device="cuda", dtype=torch.bfloat16 if quant else dtype).to(dtype)
    scales = torch.full((T, G, -(-N // 128)), -1.0, device="cuda") if quant else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.fp8_block_matmul(x, xs, B.Fp8Weights(w, ws), out, scales, status=status)
    assert B.read_device_status(status)[0] == B.OK
    wd = w.double() * ws.double().repeat_interleave(128, 1)[:, :N]
    step = max(1, (1 << 25) // max(G * N, G * K))
    for t in range(0, T, step):
        xd = x[t:t + step].double() * xs[t:t + step].double()
        y, mag = torch.einsum("tgk,gnk->tgn", xd, wd), torch.einsum("tgk,gnk->tgn", xd.abs(), wd.abs())
        err = mag * (K + 3) * 2.0 ** -23                            # k additions, the scales' product and its use
        got = out[t:t + step].double()
        if not quant:
            assert bool(((got - y).abs() <= err + (y.abs() + err) * torch.finfo(dtype).eps / 2).all())
            continue
        s = scales[t:t + step].double()
        pad = torch.nn.functional.pad(y.abs(), (0, -N % 128)).unflatten(-1, (-1, 128)).amax(-1)
        worst = torch.nn.functional.pad(err, (0, -N % 128)).unflatten(-1, (-1, 128)).amax(-1)
        # a block of zeros has scale 1; one whose sums may be zeros within their error, either
        close = (s - torch.where(pad > 0, pad / 448, 1.0)).abs() <= worst / 448 + pad / 448 * 2.0 ** -23
        off = ~(close | ((s == 1) & (pad <= worst)))
        assert not bool(off.any()), (s[off][:5], pad[off][:5], worst[off][:5])
        full = s.repeat_interleave(128, -1)[..., :N]
        # half a step of the code, of its value or of the smallest step
        assert bool(((got * full - y).abs() <= err + torch.maximum((y.abs() + err) * (2.0 ** -4 + 2.0 ** -20), full * 2.0 ** -10 * (1 + 2.0 ** -20))).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,G,N", [(2 ** 24, 1, 8), (2 ** 24, 1, 3), (1, 1, 2 ** 24), (70, 1, 2 ** 24 - 1), (1, 65535, 8), (70, 65535, 5), (300, 65535, 1)])
def test_product_of_the_most_tokens_columns_and_groups(T, G, N, dtype):
    product_against_doubles(T, G, N, 16, dtype, N)


@pytest.mark.parametrize("cols,block_rows", [(1, 1), (8, 1), (1, 128), (8, 128)])
def test_quant_of_the_most_rows(cols, block_rows):
    """2^31 - 1 blocks of 1 x 128."""
    rows = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(cols)
    p = torch.randn((1024, cols), generator=g, device="cuda").bfloat16()           # repeated down the rows
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    whole = rows // 1024 * 1024
    x[:whole].view(-1, 1024, cols).copy_(p.expand(whole // 1024, 1024, cols))
    x[whole:] = p[:rows - whole]
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-rows // block_rows), 1), -3.0, device="cuda")
    B.fp8_block_quant(x, codes, scales, block_rows=block_rows)
    del x
    v = p.float()
    s = v.view(-1, block_rows * cols).abs().amax(1) / torch.full((1024 // block_rows,), 448.0, device="cuda")
    want = (v.view(-1, block_rows * cols) / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(1024, cols)
    for a in range(0, whole, 1 << 27):
        part = codes[a:min(a + (1 << 27), whole)].view(-1, 1024, cols)
        assert bool((part == want).all())
    per = 1024 // block_rows
    assert bool((scales[:whole // block_rows].view(-1, per) == s).all())
    if block_rows == 1:
        assert torch.equal(codes[whole:], want[:rows - whole]) and torch.equal(scales[whole:, 0], s[:rows - whole])
