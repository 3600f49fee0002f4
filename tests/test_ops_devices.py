"""Handles and their operands on different devices are refused before any
launch; no GPU needed."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

from test_ops_refusals import fake

I32, I64 = torch.int32, torch.int64


def tables(monkeypatch, device):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device)
    f = lambda *shape, dtype=I32: fake(*shape, dtype=dtype, device=device)  # noqa: E731
    group = B.TableGroup(ratio=1, window=128, num_pages=8, owned=f(2, 4), table=f(2, 4), ring=f(16), pool_in=f(2, dtype=I64), pool_out=f(2, dtype=I64), slots=f(4, dtype=I64))
    return B.BatchTables([group], offsets=f(3), ctx_len=f(2), positions=f(4), seqs=f(4), row_ctx=f(4), status=f(1))


@pytest.mark.parametrize("made_on,built_on", [(0, 1), (1, 0)])
def test_tables_are_built_where_their_buffers_live(monkeypatch, made_on, built_on):
    t = tables(monkeypatch, made_on)
    calls = []
    t._call = lambda *a: calls.append(a) or 0
    # the lengths' device and the current one agree, the buffers' is another
    monkeypatch.setattr(torch.cuda, "current_device", lambda: built_on)
    lengths = [fake(2, dtype=I32, device=built_on) for _ in range(2)]
    with pytest.raises(ValueError, match="cuda:%d" % made_on):
        t.build(*lengths, stream=0)
    # the lengths where the buffers are, another device current
    lengths = [fake(2, dtype=I32, device=made_on) for _ in range(2)]
    with pytest.raises(ValueError, match="current device"):
        t.build(*lengths, stream=0)
    assert not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: made_on)
    t.build(*lengths, stream=0)
    assert len(calls) == 1
    with pytest.raises(ValueError, match="current device"):
        t.build(lengths[0], fake(2, dtype=I32, device=built_on), stream=0)
    assert len(calls) == 1


def test_tables_without_any_buffer_of_their_own_device(monkeypatch):
    """Buffers of two devices are refused when the handle is made."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f = lambda *shape, dtype=I32, device=0: fake(*shape, dtype=dtype, device=device)  # noqa: E731
    group = B.TableGroup(ratio=1, num_pages=8, owned=f(2, 4), table=f(2, 4, device=1), ring=f(16), pool_in=f(2, dtype=I64), pool_out=f(2, dtype=I64))
    with pytest.raises(ValueError, match="current device"):
        B.BatchTables([group])


def test_product_where_its_weights_live(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    w = B.Fp8Weights(fake(200, 256, dtype=torch.uint8), fake(2, 2))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="weights.*cuda:0"):
        B.fp8_block_matmul(fake(3, 256, dtype=torch.uint8, device=1), fake(3, 2, device=1), w, fake(3, 200, device=1), stream=0)
