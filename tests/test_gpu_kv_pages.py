"""Pages of the KV cache handed out on the GPU (gdn_kv_pages_grow, _trim), against
the plain Python oracle.  Everything is a whole number and has to be equal."""
import random

import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from oracle.pages_oracle import PagesOracle

pytestmark = pytest.mark.gpu
KEEP = -77  # what the outputs hold where nothing is written


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Both:
    """A cache's pages on the GPU and in the oracle."""

    def __init__(self, n_slots, n_pages, max_pages, page, host_checks=False, seed=0):
        self.kv = abi.KVCache.empty(1, n_slots, n_pages, max_pages, page, 1, 1, 64,
                                    host_checks=host_checks)
        order = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
        self.book = abi.KVPages(self.kv, i32([0] * n_slots), torch.from_numpy(order).cuda(),
                                i32([n_pages]))
        self.ref = PagesOracle(np.full((n_slots, max_pages), -1), [0] * n_slots, order, n_pages,
                               page)

    def grow(self, slots, pos, lens=None, cu=None, total=None, stream=None, tokens=True):
        if lens is not None:
            cu = np.concatenate([[0], np.cumsum(lens)])
        if total is None:
            total = len(slots) if cu is None else int(cu[-1])
        positions, rows = i32([KEEP] * total), i32([KEEP] * total).long()
        granted = i32([KEEP] * len(slots))
        want_p, want_r = np.full(total, KEEP), np.full(total, KEEP)
        abi.gdn_kv_pages_grow(self.kv, self.book, i32(slots), i32(pos),
                              None if cu is None else i32(cu), positions=positions, rows=rows,
                              granted=granted, stream=stream)
        want_g = self.ref.grow(slots, pos, cu, total, want_p, want_r)
        torch.cuda.synchronize()
        assert granted.tolist() == want_g
        if tokens:
            assert np.array_equal(positions.cpu().numpy(), want_p)
            assert np.array_equal(rows.cpu().numpy(), want_r)
        self.same()
        return want_g

    def trim(self, slots, lens, stream=None):
        abi.gdn_kv_pages_trim(self.kv, self.book, i32(slots), i32(lens), stream=stream)
        self.ref.trim(slots, lens)
        self.same()

    def same(self):
        assert np.array_equal(self.kv.page_table.cpu().numpy(), self.ref.table)
        assert self.book.held.tolist() == self.ref.held
        assert self.book.n_free.item() == self.ref.n_free
        top = max(0, min(self.ref.n_free, len(self.ref.free)))
        assert self.book.free_pages.tolist()[:top] == self.ref.free[:top]
        assert abi.gdn_kv_get_error(self.kv) == self.ref.err
        self.ref.err = 0

    def all_pages_once(self):
        table = self.kv.page_table.cpu().numpy()
        ids = [x for s, h in enumerate(self.book.held.tolist()) for x in table[s, :h]]
        ids += self.book.free_pages.tolist()[:self.book.n_free.item()]
        assert sorted(ids) == list(range(len(self.ref.free)))


@pytest.mark.parametrize("n_slots,n_pages,max_pages,page", [
    (1, 1, 1, 16), (3, 40, 20, 16), (64, 500, 33, 64), (1030, 9000, 40, 32), (2500, 6000, 9, 128)])
def test_rounds_of_growing_and_trimming(n_slots, n_pages, max_pages, page):
    """Requests that start, decode, lose drafts and end, with too few pages now and then."""
    rnd = random.Random(n_slots)
    b = Both(n_slots, n_pages, max_pages, page, seed=n_slots)
    lens = [0] * n_slots
    for _ in range(12):
        slots = rnd.sample(range(n_slots), rnd.choice([n_slots, max(1, n_slots // 2)]))
        room = max_pages * page
        kind = rnd.choice(["step", "prompts", "prompts", "trim", "end"])
        if kind in ("step", "prompts"):
            most = 1 if kind == "step" else page * max(2, n_pages // max(4, n_slots // 2))
            new = [min(room - lens[s], rnd.randint(0 if kind == "prompts" else 1, most))
                   for s in slots]
            if kind == "step" and all(x == 1 for x in new):
                got = b.grow(slots, [lens[s] for s in slots])
            else:
                got = b.grow(slots, [lens[s] for s in slots], new)
            for s, x, g in zip(slots, new, got):
                lens[s] += x if g else 0
        else:
            for s in slots:
                lens[s] = 0 if kind == "end" else rnd.randint(0, lens[s])
            b.trim(slots, [lens[s] for s in slots])
        b.all_pages_once()
    b.trim(range(n_slots), [0] * n_slots)
    assert b.book.n_free.item() == n_pages
    b.all_pages_once()


def test_many_tokens_take_many_blocks():
    """150 000 tokens in uneven sequences, and back to where it was."""
    rnd = random.Random(5)
    lens = [rnd.randint(0, 4000) for _ in range(70)] + [8192]
    b = Both(75, sum(-(-x // 16) for x in lens) + 3, 512, 16)
    slots = rnd.sample(range(75), 71)
    free = b.book.free_pages.clone()
    assert all(b.grow(slots, [0] * 71, lens))
    b.all_pages_once()
    b.trim(slots, [0] * 71)
    assert torch.equal(b.book.free_pages, free)


def test_more_sequences_than_a_round_over_many_blocks():
    lens = [random.Random(i).randint(0, 60) for i in range(3001)]
    b = Both(3001, 6000, 8, 16)
    slots = list(reversed(range(3001)))
    got = b.grow(slots, [0] * 3001, lens)
    assert 0 < got.count(0) < 1500  # the pages end before the sequences do
    b.all_pages_once()
    b.grow(slots, [x if g else 0 for x, g in zip(lens, got)])
    b.trim(slots, [x // 2 for x in lens])
    b.all_pages_once()


def test_first_come_first_served():
    """3 pages: the second sequence does not fit, the third would, the fourth needs none."""
    b = Both(4, 4, 4, 16)
    assert b.grow([3], [0], [5]) == [1]
    assert b.grow([0, 1, 2, 3], [0, 0, 0, 5], [32, 40, 3, 11]) == [1, 0, 0, 1]
    assert b.grow([1, 2], [0, 0], [16, 0]) == [1, 1]
    assert b.book.n_free.item() == 0
    assert b.grow([2], [0]) == [0]
    b.trim([0], [17])
    b.trim([0], [16])
    assert b.grow([2], [0]) == [1]


def test_slots_that_hold_more_or_fewer_pages_than_their_position():
    b = Both(2, 20, 10, 16)
    b.grow([0], [40], [1])          # pages for the positions before it too
    assert b.book.held.tolist() == [3, 0]
    b.grow([0], [0], [5])           # fewer tokens than pages: nothing to do
    assert b.book.held.tolist() == [3, 0]


def test_bad_entries_are_skipped_and_change_nothing_else():
    b = Both(8, 40, 4, 16)
    b.grow([0, 1, 2], [0, 0, 0], [20, 30, 5])
    # slots out of range, named twice; a position below zero; more than a slot holds
    b.grow([-1, 8, 3, 3, 4, 5, 6, 7], [0, 0, 0, 0, -1, 60, 0, 0], [3, 3, 3, 3, 3, 5, 65, 7])
    b.all_pages_once()
    b.trim([1, 1, 9, 2, 0], [0, 0, 0, -3, 7])
    b.all_pages_once()
    # offsets that run backwards (two sequences claim tokens: theirs are not specified), past the
    # end, below zero; tokens of no sequence
    b.grow([3, 4, 5], [0, 0, 0], cu=[4, 9, 6, 11], total=20, tokens=False)
    b.grow([3, 4], [20, 20], cu=[0, 5, 30], total=20)
    b.grow([3, 4], [20, 20], cu=[-4, 5, 8], total=20)
    b.all_pages_once()


@pytest.mark.parametrize("held", [-1, 5])
def test_a_count_that_cannot_be(held):
    b = Both(3, 12, 4, 16)
    b.grow([0, 1], [0, 0], [20, 20])
    b.book.held[1] = held
    b.ref.held[1] = held
    b.grow([0, 1, 2], [20, 20, 0], [30, 30, 30])
    b.trim([0, 1, 2], [0, 0, 0])


@pytest.mark.parametrize("n_free", [-1, 13, 2 ** 31 - 1])
def test_a_number_of_free_pages_that_cannot_be(n_free):
    b = Both(3, 12, 4, 16)
    b.grow([0, 1], [0, 0], [20, 20])
    keep = b.book.n_free.item()
    b.book.n_free.fill_(n_free)
    b.ref.n_free = n_free
    b.grow([0, 2], [20, 0], [3, 30])
    b.trim([0, 1, 2], [0, 0, 0])
    b.book.n_free.fill_(keep)
    b.ref.n_free = keep
    b.all_pages_once()


def test_pages_given_back_twice_are_not():
    """A free list that is nearly full cannot take what the counts say: nothing moves."""
    b = Both(2, 4, 4, 16)
    b.grow([0], [0], [64])
    b.book.n_free.fill_(1)
    b.ref.n_free = 1
    b.trim([0], [0])
    assert b.book.held.tolist() == [4, 0]


def test_an_invalid_page_of_the_callers():
    b = Both(2, 12, 4, 16)
    b.grow([0, 1], [0, 0], [20, 20])
    b.kv.page_table[0, 0] = 99
    b.ref.table[0, 0] = 99
    b.grow([0, 1], [10, 10], [30, 30])


def test_captured_once_and_replayed():
    """The same two calls on other lengths each time, from one graph, on its own stream."""
    b = Both(5, 30, 6, 16)
    slots, pos, cu = [4, 0, 2], i32([0, 0, 0]), i32([0, 0, 0, 0])
    total, ids, lens = 64, i32(slots), i32([0, 0, 0])
    positions, rows, granted = i32([KEEP] * total), i32([KEEP] * total).long(), i32([KEEP] * 3)

    def both():
        abi.gdn_kv_pages_trim(b.kv, b.book, ids, lens)
        abi.gdn_kv_pages_grow(b.kv, b.book, ids, pos, cu, positions=positions, rows=rows,
                              granted=granted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    b.same()
    rnd = random.Random(2)
    have = [0, 0, 0]
    for _ in range(6):
        keep = [rnd.randint(0, x) for x in have]
        new = [rnd.randint(0, min(21, 96 - k)) for k in keep]
        offs = [0, *np.cumsum(new).tolist()]
        lens.copy_(i32(keep)), pos.copy_(i32(keep)), cu.copy_(i32(offs))
        positions.fill_(KEEP), rows.fill_(KEEP)
        graph.replay()
        torch.cuda.synchronize()
        want_p, want_r = np.full(total, KEEP), np.full(total, KEEP)
        b.ref.trim(slots, keep)
        want = b.ref.grow(slots, keep, offs, total, want_p, want_r)
        b.same()
        assert granted.tolist() == want
        assert np.array_equal(positions.cpu().numpy(), want_p)
        assert np.array_equal(rows.cpu().numpy(), want_r)
        have = [k + n if g else k for k, n, g in zip(keep, new, want)]


def test_another_stream():
    b = Both(3, 12, 4, 16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.grow([0, 1], [0, 0], [20, 20])
    b.trim([0], [3], stream=s)


def test_every_output_may_be_missing():
    b = Both(3, 12, 4, 16)
    abi.gdn_kv_pages_grow(b.kv, b.book, i32([2, 0]), i32([0, 0]), i32([0, 20, 50]), 50)
    b.ref.grow([2, 0], [0, 0], [0, 20, 50], 50, np.zeros(50), np.zeros(50))
    b.same()
    abi.gdn_kv_pages_grow(b.kv, b.book, i32([]), i32([]))
    abi.gdn_kv_pages_trim(b.kv, b.book, i32([]), i32([]))
    b.same()


def test_a_call_without_any_token():
    b = Both(3, 12, 4, 16)
    b.grow([0, 1], [0, 0], [20, 20])
    assert b.grow([1, 0, 2], [20, 3, 0], [0, 0, 0]) == [1, 1, 1]


def test_host_checks_refuse_before_anything_moves():
    b = Both(4, 12, 4, 16, host_checks=True)
    b.grow([0, 1], [0, 0], [20, 20])

    def refused(name, call, *args, **kw):
        with pytest.raises(abi.GDNError) as e:
            call(b.kv, b.book, *args, **kw)
        assert e.value.name == name
        b.same()
    grow, trim = abi.gdn_kv_pages_grow, abi.gdn_kv_pages_trim
    refused("GDN_ERR_DUP_SLOT", grow, i32([2, 2]), i32([0, 0]))
    refused("GDN_ERR_SLOT", grow, i32([2, 4]), i32([0, 0]))
    refused("GDN_ERR_SIZE", grow, i32([2]), i32([64]))
    refused("GDN_ERR_SIZE", grow, i32([2]), i32([-1]))
    refused("GDN_ERR_SIZE", grow, i32([2, 3]), i32([0, 0]), i32([0, 5, 3]), 3)
    refused("GDN_ERR_SIZE", grow, i32([2, 3]), i32([0, 0]), i32([0, 5, 9]), 10)
    refused("GDN_ERR_DUP_SLOT", trim, i32([0, 0]), i32([0, 0]))
    refused("GDN_ERR_SIZE", trim, i32([0]), i32([-1]))
    b.book.n_free.fill_(10)  # 8 are free, 4 held: one page would be there twice
    refused_free = b.ref.n_free
    b.ref.n_free = 10
    refused("GDN_ERR_SIZE", trim, i32([0, 1]), i32([0, 0]))
    b.ref.n_free = refused_free


@pytest.mark.parametrize("page", [16, 128])
def test_a_cache_grown_on_the_gpu_reads_and_attends_like_one_laid_out_before(page):
    """The run that the calls are for: grow, append, attend, a draft rejected, grow again."""
    gen = torch.Generator(device="cuda").manual_seed(page)
    n, h_q, h_kv, d = 3, 4, 2, 64
    slots, prompt, drafts, kept = [2, 0, 3], [70, 1, 129], 4, [1, 4, 2]
    own = abi.KVCache.empty(1, 4, 40, 16, page, h_q, h_kv, d)
    book = abi.KVPages(own)
    fixed = abi.KVCache.empty(1, 4, 64, 16, page, h_q, h_kv, d)
    fixed.page_table.copy_(torch.arange(64, dtype=torch.int32).view(4, 16))
    ids, pos = i32(slots), i32([0] * n)
    for lens in (prompt, [drafts] * n, [1] * n):
        cu = i32(np.concatenate([[0], np.cumsum(lens)]))
        total = sum(lens)
        k, v = (torch.randn(total, h_kv, d, generator=gen, device="cuda") for _ in range(2))
        q = torch.randn(total, h_q, d, generator=gen, device="cuda")
        rows = torch.empty(total, dtype=torch.int64, device="cuda")
        granted = i32([0] * n)
        abi.gdn_kv_pages_grow(own, book, ids, pos, cu, rows=rows, granted=granted)
        assert granted.tolist() == [1] * n
        out = []
        for kv in (own, fixed):
            abi.gdn_kv_append(kv, 0, ids, pos, k, v, cu_seqlens=cu)
            out.append(abi.gdn_kv_attend(kv, 0, ids, pos + i32(lens), q, cu_seqlens=cu))
        assert torch.equal(*out)
        # the rows say where the codes are
        codes = own.k[0].transpose(1, 2).reshape(-1, h_kv, d)[rows]
        back = torch.empty_like(k)
        abi.gdn_kv_read(own, 0, ids, pos, back, None, cu_seqlens=cu)
        assert torch.equal((codes == 0), (back == 0)) and torch.equal(codes > 0, back > 0)
        pos = pos + i32(lens if lens[0] != drafts else kept)
        abi.gdn_kv_pages_trim(own, book, ids, pos)
        assert book.held[ids.long()].tolist() == [-(-p // page) for p in pos.tolist()]
    assert abi.gdn_kv_get_error(own) == 0
