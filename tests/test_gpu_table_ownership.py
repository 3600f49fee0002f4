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
