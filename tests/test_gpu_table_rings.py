"""Batch tables over rings that are as long as the cache has pages: returned
pages go to the places that the step's own pages are taken from.  Whole
numbers, so every byte has to be equal."""
import random

import numpy as np
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

from _ops_ref import first_live, pages_of, tables_ref
from test_gpu_tables import ALL, Batch, OnGpu

pytestmark = pytest.mark.gpu


def tighten(b, extra=0):
    """The batch's rings cut to the number of pages (and so many more)."""
    for g in b.groups:
        (head, tail), old = g["pool"], g["ring"]
        ring = np.full(g["num_pages"] + extra, -7, dtype=np.int64)
        for p in range(head, tail):
            ring[p % len(ring)] = old[p % len(old)]
        g["ring"] = ring
    return b


def want_of(b):
    """tables_ref over rings so long that nothing is written over, folded into
    the batch's own; and whether a group's returned pages go to places of
    taken ones."""
    wide = []
    for g in b.groups:
        (head, tail), size = g["pool"], 3 * len(g["ring"])
        ring = np.full(size, -7, dtype=np.int64)
        for p in range(head, tail):
            ring[p % size] = g["ring"][p % len(g["ring"])]
        wide.append(dict(g, ring=ring))
    want, bits = tables_ref(b.computed, b.new, wide, b.max_tokens)
    over = []
    for g, w in zip(b.groups, want["groups"]):
        ring, (head, tail), (head2, tail2) = np.array(g["ring"]), g["pool"], w["pool"]
        assert tail2 - head2 <= len(ring)
        for p in range(tail, tail2):
            ring[p % len(ring)] = w["ring"][p % len(w["ring"])]
        over.append(tail2 - head > len(ring) and head2 > head)
        w["ring"] = ring
    return want, bits, over


def check(d, want, bits):
    for k, t in d.out.items():
        if t is not None:
            assert t.cpu().tolist() == want[k], k
    for i, (g, w) in enumerate(zip(d.groups, want["groups"])):
        assert np.array_equal(g["owned"].cpu().numpy(), w["owned"]), i
        assert np.array_equal(g["table"].cpu().numpy(), w["table"]), i
        assert np.array_equal(g["ring"].cpu().numpy(), w["ring"]), i
        assert g["pool_out"].cpu().tolist() == list(w["pool"]), i
        if g["slots"] is not None:
            assert g["slots"].cpu().tolist() == w["slots"], i
    assert B.read_device_status(d.status)[1] == bits


CASES = {
    "one prompt": dict(computed=[0], new=[777], kinds=ALL, spare=0),
    "first prompts": dict(computed=[0] * 40, new=[300 + 7 * i for i in range(40)], kinds=ALL, spare=0),
    "decodes beside a long prompt": dict(computed=[500, 0, 90, 4000], new=[1, 3000, 1, 1], kinds=ALL, spare=0),
    "idle and finished": dict(computed=[500, 0, 90, 4000, 64], new=[-1, 2000, 0, -1, 500], kinds=ALL, spare=0),
    "windows": dict(computed=[0, 64, 1000, 1000], new=[900, 700, 1, -1], kinds=[(1, 128), (1, 65), (1, 64), (1, 1)], spare=0),
    "odd rows": dict(computed=[0, 700, 650], new=[1513, 1, -1], kinds=ALL, stride=41, spare=0),
    "wide rows": dict(computed=[0, 70000, 3], new=[70000, 1, 40000], kinds=ALL, stride=2600, spare=0),
    "rows behind the last": dict(computed=[0, 6], new=[900, 2], kinds=ALL, max_tokens=1500, spare=0),
    "tokens past the rows": dict(computed=[0, 10, 20], new=[900, 800, 30], kinds=ALL, max_tokens=1000, spare=0),
    "counters past 32 bits": dict(computed=[100, 200], new=[1600, -1], kinds=ALL, head=(1 << 40) + 3, spare=0),
    "a few more places": dict(computed=[0, 100], new=[2000, 1500], kinds=ALL, spare=3),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("extra", [0, 1, 5])
def test_returned_pages_in_the_places_of_taken_ones(name, off, extra):
    b = tighten(Batch(seed=len(name), **CASES[name]), extra)
    want, bits, over = want_of(b)
    assert any(over) and bits in (0, B.DEV_BAD_INDEX)
    d = OnGpu(b, off=off)
    d.tables.build(d.computed, d.new)
    check(d, want, bits)


@pytest.mark.parametrize("none", ["slots", "positions"])
def test_outputs_that_are_not_asked_for(none):
    b = tighten(Batch([0, 40], [900, 400], ALL, spare=0))
    want, bits, over = want_of(b)
    d = OnGpu(b, none=(none,))
    d.tables.build(d.computed, d.new)
    check(d, want, bits)
    assert any(over)


def test_ids_out_of_range_in_such_a_ring():
    b = tighten(Batch([0, 40], [900, 400], ALL, spare=0))
    g = b.groups[0]
    for i, v in ((0, g["num_pages"]), (5, -1), (11, 2 ** 31 - 1)):
        g["ring"][(g["pool"][0] + i) % len(g["ring"])] = v
    want, bits, over = want_of(b)
    d = OnGpu(b)
    d.tables.build(d.computed, d.new)
    check(d, want, bits)
    assert over[0] and bits == B.DEV_BAD_PAGE


@pytest.mark.parametrize("seqs,seed", [(513, 1), (2500, 2)])
def test_many_sequences(seqs, seed):
    rng = random.Random(seed)
    computed = [rng.choice((0, 0, 0, rng.randrange(400))) for _ in range(seqs)]
    new = [rng.choice((200, 1, 0, -1, rng.randrange(1, 500))) for _ in range(seqs)]
    b = tighten(Batch(computed, new, ALL, seed=seed, spare=0))
    want, bits, over = want_of(b)
    assert any(over)
    d = OnGpu(b)
    d.tables.build(d.computed, d.new)
    check(d, want, bits)


def test_a_ring_that_cannot_hold_what_is_left():
    """Two pages taken, six returned: a ring of six places serves them, one of
    five does not."""
    for size in (6, 5):
        b = Batch([300, 300, 0], [-1, -1, 100], ((1, 128),), spare=0)
        g = b.groups[0]
        ring = np.full(size, -7, dtype=np.int64)
        ring[:2] = [g["ring"][p % len(g["ring"])] for p in range(*g["pool"])]
        held = sorted(int(v) for v in g["owned"].flatten() if v >= 0)
        g["ring"], g["pool"] = ring, [0, 2]
        d = OnGpu(b)
        d.tables.build(d.computed, d.new)
        status = B.read_device_status(d.status)[1]
        if size == 6:
            assert status == 0 and d.groups[0]["pool_out"].cpu().tolist() == [2, 8]
            assert sorted(d.groups[0]["ring"].cpu().tolist()) == held
        else:
            assert status == B.DEV_BAD_PAGE and d.groups[0]["pool_out"].cpu().tolist() == [0, 2]
            assert np.array_equal(d.groups[0]["ring"].cpu().numpy(), ring)
            assert bool((d.groups[0]["table"] == -1).all())


def test_a_service_with_as_many_places_as_pages():
    """Long prompts, decodes, idles and ends; each page is free or held once
    after every step, and the ring has as many places as the cache has pages."""
    rng = random.Random(3)
    S, cap = 12, 1500
    length, live = [0] * S, [False] * S
    b = tighten(Batch([0] * S, [0] * S, ALL, max_tokens=cap, stride=60, spare=300, head=0))
    d = OnGpu(b)
    overs = 0
    for step in range(60):
        new = []
        for s in range(S):
            if not live[s]:
                length[s] = 0
                new.append(rng.randrange(1, 900) if rng.random() < 0.2 else 0)
                live[s] = new[-1] > 0
            elif rng.random() < 0.2 or length[s] > 2500:
                new.append(-1)
            else:
                new.append(rng.choice((0, 1, 1, rng.randrange(1, 200))))
        while sum(max(n, 0) for n in new) > cap:
            new[max(range(S), key=lambda s: new[s])] = 1
        b.computed, b.new = list(length), new
        want, bits, over = want_of(b)
        overs += any(over)
        d.computed.copy_(torch.tensor(length))
        d.new.copy_(torch.tensor(new))
        d.tables.build(d.computed, d.new)
        check(d, want, bits)
        assert bits == 0
        for s in range(S):
            live[s], length[s] = (False, 0) if new[s] == -1 else (live[s], length[s] + new[s])
        for g, w, t in zip(b.groups, want["groups"], d.groups):
            g["owned"], g["ring"], g["pool"] = w["owned"], w["ring"], w["pool"]
            t["pool"].copy_(t["pool_out"])
            free = [int(w["ring"][i % len(w["ring"])]) for i in range(*w["pool"])]
            held = [int(w["owned"][s, j]) for s in range(S) if live[s] for j in range(first_live(length[s], g["window"]), pages_of(length[s], g["ratio"]))]
            assert sorted(free + held) == list(range(g["num_pages"]))
    assert overs > 5
