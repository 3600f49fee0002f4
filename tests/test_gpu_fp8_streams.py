"""Products and quantisations on several streams at once: all buffers are made
and filled, and the device waited for, ahead of the first call, so that the
calls are the only work in flight and overlap."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

from test_gpu_fp8_blocks import operands, values

pytestmark = pytest.mark.gpu


def outputs(n, T, G, N, dtype):
    """n outputs, filled with what no call writes, and their scales."""
    quant = dtype == torch.float8_e4m3fn
    return [(torch.full((T, G, N), 18.0, device="cuda").to(dtype), torch.full((T, G, -(-N // 128)), -1.0, device="cuda") if quant else None) for _ in range(n)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,G,N,K", [(1, 8, 1024, 2048), (32, 8, 1024, 4096), (40, 2, 300, 1392), (700, 2, 520, 528), (2100, 3, 257, 528)])
def test_products_on_streams_of_their_own(T, G, N, K, dtype):
    x, xs, w, ws = operands(T, G, N, K, 3)
    weights = B.Fp8Weights(w, ws)
    streams = [torch.cuda.Stream() for _ in range(3)]
    (first, scales), *rest = outputs(13, T, G, N, dtype)
    torch.cuda.synchronize()
    B.fp8_block_matmul(x, xs, weights, first, scales)
    torch.cuda.synchronize()
    for i, (o, s) in enumerate(rest):
        B.fp8_block_matmul(x, xs, weights, o, s, stream=streams[i % 3])
    torch.cuda.synchronize()
    for o, s in rest:
        assert torch.equal(o.view(torch.uint8), first.view(torch.uint8))
        assert s is None or torch.equal(s, scales)


def test_different_calls_on_streams_of_their_own():
    """Few and many tokens, which share no SM, and the quantiser between them."""
    shapes = [(5, 2, 640, 1024), (64, 1, 2048, 1024), (600, 1, 512, 512), (1500, 2, 520, 528)]
    jobs = []
    for i, (T, G, N, K) in enumerate(shapes):
        x, xs, w, ws = operands(T, G, N, K, 20 + i)
        jobs.append((x, xs, B.Fp8Weights(w, ws), outputs(7, T, G, N, torch.float32)))
    a = values((700, 1000), 4, torch.bfloat16).cuda()
    quants = [(torch.full((700, 1000), 0x55, dtype=torch.uint8, device="cuda"), torch.full((700, 8), -1.0, device="cuda")) for _ in range(7)]
    streams = [torch.cuda.Stream() for _ in range(len(jobs) + 1)]
    torch.cuda.synchronize()
    for x, xs, w, outs in jobs:
        B.fp8_block_matmul(x, xs, w, outs[0][0])
    B.fp8_block_quant(a, *quants[0])
    torch.cuda.synchronize()
    for r in range(1, 7):
        for (x, xs, w, outs), s in zip(jobs, streams):
            B.fp8_block_matmul(x, xs, w, outs[r][0], stream=s)
        B.fp8_block_quant(a, *quants[r], stream=streams[-1])
    torch.cuda.synchronize()
    for _, _, _, outs in jobs:
        for o, _ in outs[1:]:
            assert torch.equal(o, outs[0][0])
    for c, s in quants[1:]:
        assert torch.equal(c, quants[0][0]) and torch.equal(s, quants[0][1])
