"""Batch tables at the ends of their ranges: the most tokens, the longest
rows, counters near 2^63."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    """These buffers are tens of GB: none stay reserved for later tests."""
    yield
    torch.cuda.empty_cache()


def i32(*shape, fill=-99):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def group(ratio, window, owned, ring, free, rows, num_pages, head=0):
    """A group whose ring holds the ids `free` from the counter head on."""
    at = (head + torch.arange(free.numel(), device="cuda")) % ring.numel()
    ring[at] = free
    return B.TableGroup(ratio=ratio, window=window, num_pages=num_pages, owned=owned, table=torch.full_like(owned, -99), ring=ring,
                        pool_in=torch.tensor([head, head + free.numel()], dtype=torch.int64, device="cuda"), pool_out=torch.full((2,), -99, dtype=torch.int64, device="cuda"),
                        slots=torch.full((rows,), -99, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("window", [0, 128])
def test_the_most_tokens(window):
    """2^24 rows of six sequences; with a window and a ring as long as the
    pages, most of them go back to the ring in the same step."""
    most = 2 ** 24
    computed = torch.tensor([0, 100, 63, 0, 5, 64])
    new = torch.tensor([1, most // 2, 70, 0, most // 4, most // 4 - 71])
    assert int(new.sum()) == most
    stride = (most // 2 + 200) // 64 + 1
    before, after = (computed + 63) // 64, (computed + new + 63) // 64
    held, taken = int(before.sum()), after - before
    pages = held + int(taken.sum())
    ids = torch.randperm(pages, device="cuda", dtype=torch.int32)
    owned = i32(6, stride, fill=-1)
    at = 0
    for s in range(6):
        owned[s, :before[s]] = ids[at:at + int(before[s])]
        at += int(before[s])
    g = group(1, window, owned, i32(pages), ids[held:].clone(), most, pages, head=(1 << 33) + 7)
    out = dict(offsets=i32(7), ctx_len=i32(6), positions=i32(most), seqs=i32(most), row_ctx=i32(most))
    status = i32(1, fill=0)
    t = B.BatchTables([g], num_seqs=6, max_tokens=most, status=status, **out)
    t.build(computed.int().cuda(), new.int().cuda())
    assert B.read_device_status(status)[1] == 0
    first = torch.cumsum(new, 0) - new
    assert out["offsets"].tolist() == first.tolist() + [most] and out["ctx_len"].tolist() == (computed + new).tolist()
    at, lo = held, [max(0, int(x) - window + 1) // 64 if window else 0 for x in computed]
    back = []
    for s in range(6):
        n, c, a = int(new[s]), int(computed[s]), int(first[s])
        pos = torch.arange(c, c + n, device="cuda")
        assert torch.equal(out["positions"][a:a + n].long(), pos) and bool((out["seqs"][a:a + n] == s).all())
        assert torch.equal(out["row_ctx"][a:a + n].long(), pos + 1)
        row = owned[s]
        assert torch.equal(row[before[s]:after[s]], ids[at:at + int(taken[s])])
        at += int(taken[s])
        assert torch.equal(g.slots[a:a + n], row[pos // 64].long() * 64 + pos % 64)
        assert torch.equal(g.table[s, lo[s]:after[s]], row[lo[s]:after[s]])
        assert bool((g.table[s, :lo[s]] == -1).all()) and bool((g.table[s, after[s]:] == -1).all())
        gone = max(0, c + n - window + 1) // 64 if window else 0
        back.append(row[lo[s]:gone].clone() if gone > lo[s] else row[:0].clone())
    back = torch.cat(back)
    head, tail = g.pool_in.tolist()
    assert g.pool_out.tolist() == [head + int(taken.sum()), tail + back.numel()]
    if back.numel():
        assert torch.equal(g.ring[(tail + torch.arange(back.numel(), device="cuda")) % pages], back)


def test_the_longest_rows():
    """Rows of which the last entries lie past 2^32 bytes; one is filled to its
    end."""
    stride = (2 ** 31 - 2 ** 12) // 3 - 1
    owned = i32(3, stride, fill=-1)
    pages = stride * 64 // 64 + 3
    full = 2 ** 31 - 200
    n_full = (full + 63) // 64
    owned[2, :n_full] = torch.arange(n_full, dtype=torch.int32, device="cuda")
    g = group(1, 0, owned, i32(64), torch.arange(n_full, n_full + 40, dtype=torch.int32, device="cuda"), 400, pages)
    status, ctx, pos = i32(1, fill=0), i32(3), i32(400)
    t = B.BatchTables([g], num_seqs=3, max_tokens=400, ctx_len=ctx, positions=pos, status=status)
    t.build(torch.tensor([0, 0, full], dtype=torch.int32, device="cuda"), torch.tensor([100, 0, 199], dtype=torch.int32, device="cuda"))
    assert B.read_device_status(status)[1] == 0
    assert ctx.tolist() == [100, 0, 2 ** 31 - 1]
    assert pos.tolist() == list(range(100)) + list(range(full, full + 199)) + [-1] * 101
    after = (2 ** 31 - 1 + 63) // 64
    assert g.table[0, :2].tolist() == [n_full, n_full + 1] and torch.equal(g.table[2, :after], owned[2, :after])
    for s, a in ((0, 2), (1, 0), (2, after)):
        assert bool((g.table[s, a:] == -1).all())
    assert g.slots[:100].tolist() == [(n_full + p // 64) * 64 + p % 64 for p in range(100)]
    assert g.slots[100:299].tolist() == [int(owned[2, p // 64]) * 64 + p % 64 for p in range(full, full + 199)]


@pytest.mark.parametrize("head,served", [(2 ** 63 - 1 - 20, True), (2 ** 63 - 1 - 10, False)])
def test_counters_near_their_end(head, served):
    """Ten pages are free and five go back: a counter may reach 2^63 - 1 and
    not pass it."""
    owned = i32(2, 20, fill=-1)
    owned[0, :5] = torch.arange(5, dtype=torch.int32, device="cuda")
    g = group(1, 0, owned, i32(15), torch.arange(5, 15, dtype=torch.int32, device="cuda"), 200, 15, head=head)
    status = i32(1, fill=0)
    t = B.BatchTables([g], num_seqs=2, max_tokens=200, status=status)
    t.build(torch.tensor([300, 0], dtype=torch.int32, device="cuda"), torch.tensor([-1, 130], dtype=torch.int32, device="cuda"))
    assert B.read_device_status(status)[1] == (0 if served else B.DEV_BAD_PAGE)
    tail = head + 10
    assert g.pool_out.tolist() == ([head + 3, tail + 5] if served else [head, tail])
    assert g.table[1, :3].tolist() == ([5, 6, 7] if served else [-1] * 3)
    if served:
        assert [int(g.ring[(tail + i) % 15]) for i in range(5)] == list(range(5))
