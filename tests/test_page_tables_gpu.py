"""Block tables and slot maps built on the GPU against the same steps one
request at a time on the host: whole numbers, equal."""
import numpy as np
import pytest
import torch

from paged_kv_flash_gb300 import workloads as W
from tests import int4_ref as R
from tests.helpers import dev, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_flash_gb300 import pagedkv
    return pagedkv


class Host:
    """The requests, their pages and the ring, one request at a time."""

    def __init__(self, rng, lens, max_pages, spare, slack=0):
        self.lens = np.asarray(lens, np.int64)
        held = -(-self.lens // 16)
        self.num_pages = int(held.sum()) + spare + slack
        perm = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), max_pages), -1, np.int64)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.ring = np.full(self.num_pages, -1, np.int64)
        self.head, self.count = int(rng.integers(self.num_pages)), spare
        self.ring[(self.head + np.arange(spare)) % self.num_pages] = perm[at:at + spare]

    def device(self):
        i = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
        return dict(seq_lens=i(self.lens), block_table=i(self.table), free_ring=i(self.ring),
                    ring_state=i([self.head, self.count]))

    def step(self, new):
        cu, taken, freed, slots = [0], [0], [0], []
        tail = self.head + self.count
        cap = len(self.ring)
        for b, n in enumerate(new):
            held = -(-self.lens[b] // 16)
            if n < 0:
                for j in range(held):
                    self.ring[tail % cap] = self.table[b, j]
                    tail += 1
                self.lens[b] = 0
                taken.append(taken[-1])
                freed.append(freed[-1] + held)
                cu.append(cu[-1])
                continue
            need = -(-(self.lens[b] + n) // 16) - held
            for j in range(need):
                self.table[b, held + j] = self.ring[self.head % cap]
                self.head += 1
            for p in range(self.lens[b], self.lens[b] + n):
                slots.append(self.table[b, p // 16] * 16 + p % 16)
            self.lens[b] += n
            cu.append(cu[-1] + n)
            taken.append(taken[-1] + need)
            freed.append(freed[-1])
        self.count = tail - self.head
        self.head %= cap
        return cu, [taken, freed], slots


def eq(t, want):
    assert np.array_equal(t.cpu().numpy(), np.asarray(want, np.int32))


@pytest.mark.parametrize("B", [1, 7, 64, 1023, 1024, 1025, 5000])
@pytest.mark.parametrize("in_place", [True, False])
def test_steps_match_the_host(pk, B, in_place):
    """Several steps: mixed new lengths (none, one, many), ended and re-admitted
    requests, the ring wrapping round, the arrays updated in place or beside."""
    rng = np.random.default_rng(1000 + B)
    host = Host(rng, rng.integers(0, 70, B), max_pages=40, spare=B * 12 + 8)
    d = host.device()
    for step in range(4):
        new = rng.choice([-1, 0, 1, 1, 1, 17, 100], B) if B > 1 else np.array([[100, 1, -1, 33][step]])
        tokens = int(np.maximum(new, 0).sum())
        slots = torch.full((tokens + 5,), -9, dtype=torch.int32, device="cuda")
        offs = torch.empty((2, B + 1), dtype=torch.int32, device="cuda")
        out = {} if in_place else dict(seq_lens_out=torch.empty_like(d["seq_lens"]),
                                       ring_state_out=torch.empty_like(d["ring_state"]))
        cu, lens = pk.page_tables(d["seq_lens"], dev(new.astype(np.int32)), d["block_table"],
                                  d["free_ring"], d["ring_state"], host.num_pages, slot_map=slots,
                                  page_offsets=offs, **out)
        assert pk.poll_device_error() == pk.OK
        if not in_place:
            eq(d["seq_lens"], host.lens)                      # the inputs are left alone
            eq(d["ring_state"], [host.head, host.count])
            d["seq_lens"], d["ring_state"] = lens, out["ring_state_out"]
        hcu, hoffs, hslots = host.step(new)
        eq(cu, hcu)
        eq(offs, hoffs)
        eq(slots, hslots + [-9] * 5)
        eq(d["seq_lens"], host.lens)
        eq(d["block_table"], host.table)
        eq(d["free_ring"], host.ring)
        eq(d["ring_state"], [host.head, host.count])


@pytest.mark.parametrize("B,choices", [(2000, [-1, 0, 1, 2]), (2049, [0, 1]), (3, [2700]),
                                       (3, [2800, 0]), (900, [-1])])
def test_small_and_large_steps(pk, B, choices):
    """Either side of what one CTA does alone: many requests of few tokens, few
    of many, all of them ending."""
    rng = np.random.default_rng(1050 + B)
    host = Host(rng, rng.integers(0, 60, B), max_pages=400, spare=B * 3 + 1200)
    d = host.device()
    for _ in range(2):
        new = rng.choice(choices, B)
        tokens = int(np.maximum(new, 0).sum())
        slots = torch.full((tokens + 1,), -9, dtype=torch.int32, device="cuda")[1:]    # unaligned
        offs = torch.empty((2, B + 1), dtype=torch.int32, device="cuda")
        cu, lens = pk.page_tables(d["seq_lens"], dev(new.astype(np.int32)), d["block_table"],
                                  d["free_ring"], d["ring_state"], host.num_pages,
                                  slot_map=slots if tokens else None, page_offsets=offs)
        assert pk.poll_device_error() == pk.OK
        hcu, hoffs, hslots = host.step(new)
        for got, want in ((cu, hcu), (offs, hoffs), (slots, hslots), (lens, host.lens),
                          (d["block_table"], host.table), (d["free_ring"], host.ring),
                          (d["ring_state"], [host.head, host.count])):
            eq(got, want)


def test_the_last_free_page_and_no_slot_map(pk):
    """Exactly as many pages as are free; no slot map; a request of no tokens."""
    rng = np.random.default_rng(1100)
    host = Host(rng, [16, 0, 5], max_pages=4, spare=3)
    d = host.device()
    new = np.array([32, 0, 12], np.int32)
    cu, lens = pk.page_tables(d["seq_lens"], dev(new), d["block_table"], d["free_ring"],
                              d["ring_state"], host.num_pages)
    assert pk.poll_device_error() == pk.OK
    hcu, _, _ = host.step(new)
    eq(cu, hcu)
    eq(lens, [48, 0, 17])
    eq(d["block_table"], host.table)
    assert host.count == 0
    eq(d["ring_state"], [host.head, 0])


@pytest.mark.parametrize("what", ["pages", "slots", "table", "length", "head", "count", "ring"])
def test_a_step_that_does_not_fit_changes_nothing(pk, what):
    rng = np.random.default_rng(1200)
    host = Host(rng, [16, 30, 5, 0], max_pages=8, spare=8)
    new = np.array([17, -1, 3, 1], np.int32)
    if what == "pages":
        new[3] = 8 * 16 - 15
    if what == "table":
        new[0] = 8 * 16 - 15
    d = host.device()
    if what == "length":
        d["seq_lens"][2] = -1
    if what == "head":
        d["ring_state"][0] = host.num_pages
    if what == "count":
        d["ring_state"][1] = -1
    if what == "ring":                                        # freeing would pass the capacity
        d["ring_state"][1] = host.num_pages
        new[:] = [0, -1, 0, 0]
    slots = torch.full((3 if what == "slots" else 400,), -9, dtype=torch.int32, device="cuda")
    before = {n: t.clone() for n, t in d.items()}
    offs = torch.full((2, 5), 77, dtype=torch.int32, device="cuda")
    cu, _ = pk.page_tables(d["seq_lens"], dev(new), d["block_table"], d["free_ring"],
                           d["ring_state"], host.num_pages, slot_map=slots, page_offsets=offs)
    assert pk.poll_device_error() == pk.ERR_INVALID
    assert pk.poll_device_error() == pk.OK
    for n, t in before.items():
        assert torch.equal(d[n], t), n
    eq(cu, [0] * 5)
    eq(offs, [[0] * 5] * 2)
    assert (slots == -9).all()


def test_page_ids_outside_the_pool_are_flagged(pk):
    rng = np.random.default_rng(1300)
    host = Host(rng, [16, 20], max_pages=4, spare=4)
    d = host.device()
    d["free_ring"][(host.head + 0) % host.num_pages] = host.num_pages       # request 0's page
    slots = torch.full((3,), -9, dtype=torch.int32, device="cuda")
    pk.page_tables(d["seq_lens"], dev(np.array([2, 1], np.int32)), d["block_table"],
                   d["free_ring"], d["ring_state"], host.num_pages, slot_map=slots)
    assert pk.poll_device_error() == pk.ERR_INVALID
    eq(slots, [-1, -1, host.table[1, 1] * 16 + 4])


def test_a_captured_loop_of_steps(pk):
    """One graph of table update and 4-bit append, replayed: the state moves on
    the GPU alone, pages are taken as the sequences grow, and the pool ends as
    the host's own steps leave it."""
    rng = np.random.default_rng(1400)
    B, Hkv, steps = 5, 2, 20
    host = Host(rng, [15, 0, 16, 7, 31], max_pages=6, spare=12)
    d = host.device()
    new = dev(np.array([1, 1, 1, 0, 1], np.int32))
    cu, offs = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B + 1,), (2, B + 1)))
    slots = torch.empty(4, dtype=torch.int32, device="cuda")
    kn = W.normal_bf16(rng, (steps + 1, 4, Hkv, 128))
    vn = W.normal_bf16(rng, kn.shape)
    kd, vd = dev_bf16(kn[0]), dev_bf16(vn[0])
    pool = pk.Pool(*(torch.zeros((host.num_pages, Hkv, 1152), dtype=torch.uint8, device="cuda")
                     for _ in range(2)))

    def step():
        pk.page_tables(d["seq_lens"], new, d["block_table"], d["free_ring"], d["ring_state"],
                       host.num_pages, cu_new=cu, page_offsets=offs, slot_map=slots)
        pk.kv_append(pool, kd, vd, cu, d["block_table"], d["seq_lens"])

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()                                                # warm-up: step 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    want = [np.zeros((host.num_pages, Hkv, 1152), np.uint8) for _ in range(2)]
    for i in range(steps + 1):
        if i:
            kd.copy_(dev_bf16(kn[i]))
            vd.copy_(dev_bf16(vn[i]))
            g.replay()
            torch.cuda.synchronize()
        _, _, hslots = host.step([1, 1, 1, 0, 1])
        eq(slots, hslots)
        for pool_h, x in zip(want, (kn[i], vn[i])):
            for t, sl in enumerate(hslots):
                for h in range(Hkv):
                    R.put(pool_h, sl // 16, h, sl % 16,
                          *R.quantize(W.bits_to_float(x[t, h]).astype(np.float32)))
    assert pk.poll_device_error() == pk.OK
    eq(d["seq_lens"], host.lens)
    eq(d["block_table"], host.table)
    assert np.array_equal(pool.k.cpu().numpy(), want[0])
    assert np.array_equal(pool.v.cpu().numpy(), want[1])
