"""Batch tables step after step: what a refused step leaves, and what a
finished sequence returns."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

from _ops_ref import first_live, pages_of
from test_gpu_tables import ALL, Batch, OnGpu

pytestmark = pytest.mark.gpu


class Service:
    """A batch's buffers from step to step; the counters move along."""

    def __init__(self, seqs, kinds, **kw):
        self.b = Batch([0] * seqs, [0] * seqs, kinds, max_tokens=2048, stride=40, **kw)
        self.d = OnGpu(self.b)

    def step(self, computed, new, advance=True):
        self.d.status.zero_()
        self.d.computed.copy_(torch.tensor(computed))
        self.d.new.copy_(torch.tensor(new))
        self.d.tables.build(self.d.computed, self.d.new)
        if advance:
            for g in self.d.groups:
                g["pool"].copy_(g["pool_out"])
        return B.read_device_status(self.d.status)[1]

    def free(self, g):
        ring, (head, tail) = self.d.groups[g]["ring"].cpu().tolist(), self.d.groups[g]["pool"].cpu().tolist()
        return [ring[p % len(ring)] for p in range(head, tail)]


@pytest.mark.parametrize("tight", [False, True])
@pytest.mark.parametrize("kind", ["swa", "full", "c4"])
def test_a_step_behind_a_refused_one_shares_no_pages(kind, tight):
    """Row 0 held pages before; its next sequence's first step finds the pool
    empty, and the caller goes on as if it had been served."""
    s = Service(2, (kind,), spare=60)
    if tight:
        g = s.d.groups[0]
        ring = g["ring"].clone()
        head, tail = g["pool"].cpu().tolist()
        g["ring"][:60].copy_(torch.tensor([int(ring[p % len(ring)]) for p in range(head, tail)], dtype=torch.int32))
        g["pool"].copy_(torch.tensor([0, 60]))
        s.d.tables = B.BatchTables([B.TableGroup(ratio=g["h"].ratio, window=g["h"].window, num_pages=60, owned=g["owned"], table=g["table"], ring=g["ring"][:60],
                                                 pool_in=g["pool"], pool_out=g["pool_out"], slots=g["slots"])], num_seqs=2, max_tokens=2048, status=s.d.status, **s.d.out)
        g["ring"] = g["ring"][:60]
    ratio = s.b.groups[0]["ratio"]
    assert s.step([0, 0], [1100, 300]) == 0
    assert s.step([1100, 300], [-1, 1]) == 0
    full = s.d.groups[0]["pool"].clone()
    s.d.groups[0]["pool"][0] = s.d.groups[0]["pool"][1]                # nothing free
    assert s.step([0, 301], [1000, 0], advance=False) == B.DEV_BAD_PAGE
    assert s.d.groups[0]["owned"][0, :pages_of(1000, ratio)].eq(-1).all()
    assert s.d.groups[0]["table"][0].eq(-1).all()
    s.d.groups[0]["pool"].copy_(full)
    for _ in range(2):
        assert s.step([1000, 301], [1, 0], advance=False) == B.DEV_BAD_PAGE
        shown = [v for v in s.d.groups[0]["table"].flatten().cpu().tolist() if v >= 0]
        assert len(shown) == len(set(shown)) and shown and not set(shown) & set(s.free(0))
        assert s.d.groups[0]["table"][0, :pages_of(1000, ratio)].eq(-1).all()


def test_a_refused_step_leaves_the_entries_held_before():
    s = Service(1, ALL, spare=60)
    assert s.step([0], [300]) == 0
    held = [g["owned"].clone() for g in s.d.groups]
    for g in s.d.groups:
        g["pool"][0] = g["pool"][1]
    assert s.step([300], [400], advance=False) == B.DEV_BAD_PAGE
    for g, h, b in zip(s.d.groups, held, s.b.groups):
        n, lo = pages_of(300, b["ratio"]), first_live(300, b["window"])
        assert torch.equal(g["owned"][:, :n], h[:, :n]) and torch.equal(g["table"][:, lo:n], h[:, lo:n])
        assert g["table"][:, :lo].eq(-1).all() and g["table"][:, n:].eq(-1).all()


@pytest.mark.parametrize("kind", ["swa", "full", "c4"])
@pytest.mark.parametrize("value", [-1, 60, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("busy", [False, True])
def test_a_finished_sequence_with_an_id_out_of_range(kind, value, busy):
    """What it returns is flagged; `busy`: beside a prompt whose pages pass
    through the same places of the ring."""
    s = Service(2, (kind,), spare=60)
    assert s.step([0, 0], [1100, 0]) == 0
    g, (ratio, window) = s.d.groups[0], (s.b.groups[0]["ratio"], s.b.groups[0]["window"])
    if busy:
        # as many places as pages: the prompt takes all that are free
        ring, pool = g["ring"].cpu().tolist(), g["pool"].cpu().tolist()
        free = [ring[p % len(ring)] for p in range(*pool)]
        size = len(free) + pages_of(1100, ratio) - first_live(1100, window)
        cut = torch.full((size,), -7, dtype=torch.int32, device="cuda")
        cut[:len(free)] = torch.tensor(free, dtype=torch.int32)
        g["ring"] = cut
        g["pool"].copy_(torch.tensor([0, len(free)]))
        s.d.tables = B.BatchTables([B.TableGroup(ratio=ratio, window=window, num_pages=60, owned=g["owned"], table=g["table"], ring=cut, pool_in=g["pool"],
                                                 pool_out=g["pool_out"], slots=g["slots"])], num_seqs=2, max_tokens=2048, status=s.d.status, **s.d.out)
    last = pages_of(1100, ratio) - 1
    old = g["owned"][0, first_live(1100, window):last + 1].tolist()
    g["owned"][0, last] = value
    before = g["pool"].cpu().tolist()
    new = [-1, 1900 if busy and kind == "swa" else 0]
    assert s.step([1100, 0], new, advance=False) == B.DEV_BAD_PAGE
    head, tail = g["pool_out"].cpu().tolist()
    assert head == before[0] + pages_of(max(new[1], 0), ratio)
    back = [int(g["ring"][p % g["ring"].numel()]) for p in range(before[1], before[1] + len(old))]
    assert back == old[:-1] + [value]
    g["owned"][0, last] = old[-1]
    if not busy:
        assert s.step([1100, 0], new, advance=False) == 0


def test_a_live_sequences_returned_id_out_of_range():
    s = Service(1, ("swa",), spare=60)
    assert s.step([0], [300]) == 0
    s.d.groups[0]["owned"][0, first_live(300, 128)] = 99
    assert s.step([300], [100]) == B.DEV_BAD_PAGE
