"""Page operations against plain lists of whole numbers: exact."""

import random

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

BAD_INDEX, NO_PAGES = 5, 6


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class State:
    """A random pool on the GPU and its restatement."""

    def __init__(self, rows, max_len, pages, seed, empty_rows=0, width=None):
        rng = random.Random(seed)
        lens = [rng.randint(0, max_len) for _ in range(rows)] + [0] * empty_rows
        width = width or -(-max_len // 64) + 3
        perm = list(range(pages))
        rng.shuffle(perm)
        table = np.full((rows + empty_rows, width), -1, dtype=np.int32)
        ref = np.zeros(pages, dtype=np.int32)
        for r, n in enumerate(lens):
            for j in range(-(-n // 64)):
                table[r, j] = perm.pop()
                ref[table[r, j]] = 1
        self.ref, self.table, self.lens = i32(ref), torch.from_numpy(table).cuda(), i32(lens)
        self.host = so.Pool(ref, table, lens)
        self.status = i32([0])

    def same(self):
        assert self.ref.tolist() == self.host.ref
        assert self.lens.tolist() == self.host.lens
        assert self.table.tolist() == self.host.table
        code = int(self.status)
        assert (code != 0) == (self.host.bad or self.host.empty)
        if code:
            assert (code == BAD_INDEX and self.host.bad) or (code == NO_PAGES and self.host.empty)

    def grow(self, rows, new):
        self.host.grow(rows, new)
        mla.cache_grow(self.ref, self.table, self.lens, i32(rows), i32(new), status=self.status)
        self.same()

    def fork(self, parents, children):
        want = self.host.fork(parents, children)
        got = mla.cache_fork(self.ref, self.table, self.lens, i32(parents), i32(children), status=self.status)
        assert [tuple(p) for p in got.tolist()] == want
        self.same()

    def free(self, rows):
        self.host.free(rows)
        mla.cache_free(self.ref, self.table, self.lens, i32(rows), status=self.status)
        self.same()

    def compact(self):
        want = self.host.compact()
        pairs, count = mla.cache_compact(self.ref, self.table, self.lens, status=self.status)
        got = [tuple(p) for p in pairs.tolist()]
        assert int(count) == len(want) and got[:len(want)] == want
        assert all(p == (-1, -1) for p in got[len(want):])
        self.same()


@pytest.mark.parametrize("pages", [64, 1023, 8192, 8193, 20000])
def test_grow_takes_the_lowest_free_pages(pages):
    s = State(9, 250, pages, seed=pages)
    s.grow([3, 0, 8], [64, 1, 130])
    s.grow([5], [0])
    s.grow(list(range(9)), [7 * i for i in range(9)])


def test_grow_many_rows():
    s = State(3000, 64, 9000, seed=1, width=5)
    s.grow(list(range(0, 3000, 2)), [i % 140 for i in range(1500)])
    s.grow(list(range(3000)), [1] * 3000)


def test_grow_until_the_pool_is_empty():
    s = State(6, 100, 20, seed=2, width=30)
    free = s.host.ref.count(0)
    s.grow([0], [64 * (free - 1)])
    assert not s.host.empty
    # the first needs none, the second more than is left, the third none, the fourth one
    s.grow([1, 2, 3, 4], [0, 64 * 5, 0, 64])
    assert s.host.empty and s.host.ref.count(0) >= 1


@pytest.mark.parametrize("rows,new", [([0, 1, 0], [5, 5, 5]), ([-1, 2], [5, 5]), ([7, 2], [5, 5]), ([1, 2], [-1, 5]),
                                      ([1, 2], [10 ** 6, 5]), ([1, 2], [2 ** 31 - 1, 5])])
def test_grow_refuses_bad_entries_only(rows, new):
    s = State(4, 200, 100, seed=3)
    s.grow(rows, new)
    assert s.host.bad


def test_fork_shares_full_pages_and_copies_the_tail():
    s = State(5, 400, 200, seed=4, empty_rows=9)
    s.fork([0, 1, 1, 1, 4], [5, 6, 7, 8, 9])
    s.fork([5, 2], [10, 11])          # a fork of a fork
    s.grow([5, 6, 7], [1, 64, 100])
    s.free([1, 6])
    s.fork([7], [1])                  # into a freed row
    s.free(list(range(14)))
    assert not any(s.host.ref)


@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 128])
def test_fork_lengths(length):
    s = State(1, 0, 10, seed=5, empty_rows=3, width=4)
    s.grow([0], [length])
    s.fork([0, 0], [1, 3])


@pytest.mark.parametrize("parents,children", [([0, 0], [4, 4]), ([0, 4], [4, 5]), ([0, 1], [1, 4]), ([0, 0], [0, 4]),
                                              ([-1, 0], [4, 5]), ([9, 0], [4, 5]), ([0, 0], [6, 5]),
                                              ([0, 0], [-2, 5])])
def test_fork_refuses_bad_entries_only(parents, children):
    s = State(4, 200, 100, seed=6, empty_rows=2)
    s.grow([0, 1], [65, 65])  # neither is empty
    s.fork(parents, children)
    assert s.host.bad


def test_fork_without_pages():
    s = State(1, 0, 5, seed=7, empty_rows=6, width=8)
    s.grow([0], [100])
    s.fork([0] * 5, [1, 2, 3, 4, 5])
    assert s.host.empty and s.host.lens == [100, 100, 100, 100, 0, 0, 0]


def test_free_twice_and_bad_rows():
    s = State(4, 200, 60, seed=8)
    s.free([1, 1, 1])
    assert not s.host.bad
    s.free([1])
    s.free([7, 0, -1])
    assert s.host.bad


def test_free_reports_pages_that_are_free_already():
    s = State(2, 200, 30, seed=9, empty_rows=1)
    s.host.lens[2], s.host.table[2][0] = 40, s.host.ref.index(0)
    s.lens, s.table = i32(s.host.lens), torch.tensor(s.host.table, dtype=torch.int32, device="cuda")
    s.free([2])
    assert s.host.bad


@pytest.mark.parametrize("pages,rows,max_len", [(1, 0, 0), (2, 1, 64), (3, 2, 64), (100, 6, 300), (4096, 40, 900),
                                                (4097, 200, 900), (13000, 400, 1500)])
def test_compact(pages, rows, max_len):
    s = State(max(rows, 1), max_len, pages, seed=pages)
    if rows > 3:
        s.free([0])
        s.fork([1, 2], [0] + ([] if rows < 4 else [0]))  # the second is refused: same child
        s.status.zero_()
        s.host.bad = False
    s.compact()
    live = [c for c in s.host.ref if c]
    assert s.host.ref[:len(live)] == live
    s.compact()  # nothing left to move


def test_compact_full_and_empty_pools():
    s = State(1, 0, 50, seed=11)
    s.compact()
    s.grow([0], [64 * 3])
    s.compact()
    s = State(1, 64 * 50, 50, seed=12, width=60)
    s.grow([0], [64 * s.host.ref.count(0)])
    s.compact()


def test_compact_reports_entries_that_name_free_pages():
    s = State(3, 200, 40, seed=13)
    s.host.lens[0] = s.host.lens[0] // 64 * 64 + 1  # its last entry: a free page, or none
    row = s.host.table[0]
    row[(s.host.lens[0] - 1) // 64] = -1
    s.lens, s.table = i32(s.host.lens), torch.tensor(s.host.table, dtype=torch.int32, device="cuda")
    s.compact()
    assert s.host.bad


# ------------------------------------------------------------------ copy


def pool_of(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype == torch.uint8:
        return torch.randint(0, 256, shape, dtype=dtype, device="cuda", generator=g)
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def check_copy(pool, pairs, layered, count=None):
    want = pool.clone()
    flat = want if layered else want[None]
    used = pairs if count is None else pairs[:count]
    done, bad = so.copy_pairs(used, flat.shape[1])
    before = flat.clone()
    for a, b in done:
        flat[:, b] = before[:, a]
    status = i32([0])
    mla.cache_copy_pages(pool, i32(pairs).reshape(-1, 2), None if count is None else i32([count]), layered, status)
    assert torch.equal(pool, want)
    assert int(status) == (BAD_INDEX if bad else 0)


@pytest.mark.parametrize("shape,dtype,layered", [
    ((40, 64, 576), torch.bfloat16, False), ((40, 64, 656), torch.uint8, False), ((3, 40, 64, 656), torch.uint8, True),
    ((2, 40, 64, 576), torch.float16, True), ((40, 64, 2, 576), torch.bfloat16, False), ((5, 40, 8), torch.float32, True)])
def test_copy_pages(shape, dtype, layered):
    pool = pool_of(shape, dtype, 1)
    check_copy(pool, [(0, 39), (3, 5), (-1, -1), (3, 6), (7, 7), (30, 1)], layered)


def test_copy_layers_with_a_gap():
    whole = pool_of((3, 21, 64, 576), torch.bfloat16, 2)
    keep = whole[:, 20].clone()
    check_copy(whole[:, :20], [(1, 2), (3, 4)], True)
    assert torch.equal(whole[:, 20], keep)


@pytest.mark.parametrize("pairs", [[(0, 1), (2, 1)], [(0, 1), (1, 2)], [(0, 1), (1, 0)], [(0, 40)], [(-1, 3), (4, 5)],
                                   [(5, -7), (4, 6)], [(1, 1), (0, 1)], [(0, 1), (0, 1), (0, 2)]])
def test_copy_refuses_what_would_depend_on_order(pairs):
    check_copy(pool_of((2, 40, 64, 16), torch.bfloat16, 3), pairs, True)


@pytest.mark.parametrize("count", [0, 1, 5, 99])
def test_copy_count_on_the_device(count):
    check_copy(pool_of((60, 64, 16), torch.bfloat16, 4), [(i, 30 + i) for i in range(8)], False, count)


def test_copy_many_pairs():
    n = 3000
    order = torch.randperm(2 * n, generator=torch.Generator().manual_seed(5)).tolist()
    check_copy(pool_of((2, 2 * n, 64, 4), torch.float16, 6), list(zip(order[:n], order[n:])), True)


def test_copy_tens_of_thousands_of_pairs():
    """Blocks that judge more pairs than one pass over the list takes; a few of them refused."""
    n, pages = 50000, 100100
    g = torch.Generator().manual_seed(7)
    pairs = torch.randperm(pages, generator=g)[:2 * n].reshape(n, 2).int()
    pairs[20000, 1] = pairs[31, 1]       # a target named before: the later pair is refused
    pairs[49999] = pairs[77]             # the same pair again
    pairs[12345, 1] = pairs[48000, 0]    # a target that another pair reads
    pairs[33333, 1] = pages              # outside the pool
    refused = torch.tensor([20000, 49999, 12345, 33333])
    pool = torch.randint(0, 256, (pages, 16), dtype=torch.uint8, generator=g).cuda()
    keep = torch.ones(n, dtype=torch.bool)
    keep[refused] = False
    done = pairs[keep].long().cuda()
    want = pool.clone()
    want[done[:, 1]] = pool[done[:, 0]]
    status = i32([0])
    mla.cache_copy_pages(pool, pairs.cuda(), status=status)
    assert torch.equal(pool, want) and int(status) == BAD_INDEX


def test_copy_past_32_bits():
    pages = (1 << 32) // (64 * 1152) + 40
    pool = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    pool[pages - 1] = 3
    mla.cache_copy_pages(pool, i32([[pages - 1, pages - 2], [pages - 1, 2]]))
    assert torch.all(pool[pages - 2] == 3) and torch.all(pool[2] == 3)
    pool[pages - 2:] = 0
    pool[2] = 0
    assert not pool.any()


@pytest.mark.parametrize("length", [-1, -2 ** 31, 7 * 64 + 1, 10 ** 6, 2 ** 31 - 1])
def test_free_leaves_a_row_whose_length_is_out_of_range(length):
    """Such an entry is reported and its row left as it was; entries behind a length are not read."""
    s = State(3, 200, 60, seed=20)
    assert len(s.host.table[0]) == 7
    s.host.lens[1] = length
    s.host.table[1][5:] = s.host.table[0][:1] + s.host.table[2][:1]  # stale: pages of the other rows
    s.lens, s.table = i32(s.host.lens), i32(s.host.table)
    s.free([1, 0, 1])
    assert s.host.bad and s.host.lens[1] == length and s.host.lens[0] == 0


@pytest.mark.parametrize("page", [-1, 40, 10 ** 6, "free"])
@pytest.mark.parametrize("where", [0, 1, 3])  # full pages, the partly filled last one
def test_fork_refuses_a_parent_with_a_bad_page(where, page):
    """A parent that names a page outside the pool, or a free one, forks into nothing; the other entries are
    served, with the lowest free pages."""
    s = State(2, 0, 40, seed=21, empty_rows=5, width=6)
    s.grow([0, 1], [200, 150])
    s.host.table[0][where] = s.host.ref.index(0) if page == "free" else page
    s.table = i32(s.host.table)
    s.fork([0, 1, 0, 1], [3, 4, 5, 6])
    assert s.host.bad and s.host.lens == [200, 150, 0, 0, 150, 0, 150]
    assert s.host.table[3] == s.host.table[5] == [-1] * 6


def test_copy_long_list():
    """Hundreds of thousands of pairs, thousands of them refused: a target named before, a target that another
    pair reads, the same pair again, pages outside the pool."""
    n, pages = 300000, 700001
    g = torch.Generator().manual_seed(8)
    pairs = torch.randperm(pages, generator=g)[:2 * n].reshape(n, 2).int()
    at = torch.randperm(n, generator=g)
    pairs[at[:2000], 1] = pairs[at[5000:7000], 1]    # the later of two is refused
    pairs[at[2000:4000], 1] = pairs[at[7000:9000], 0]
    pairs[at[4000:4100]] = pairs[at[9000:9100]]
    pairs[at[4100:4200], 1] = pages + 5
    pairs[at[4200:4300], 0] = -3
    pairs[at[4300:4400]] = -1
    pairs[at[4400:4500], 0] = pairs[at[4400:4500], 1]  # a page onto itself: skipped, but it is the first of its target
    x, y = pairs[:, 0].numpy().astype(np.int64), pairs[:, 1].numpy().astype(np.int64)
    first = np.full(pages + 6, n)
    np.minimum.at(first, y[y >= 0], np.nonzero(y >= 0)[0])
    read = np.zeros(pages + 6, dtype=bool)
    read[x[(x >= 0) & (x != y)]] = True
    skip = ((x < 0) & (y < 0)) | (x == y)
    good = (x >= 0) & (y >= 0) & (x < pages) & (y < pages)
    good &= (first[np.maximum(y, 0)] == np.arange(n)) & ~read[np.maximum(y, 0)]
    done = torch.from_numpy(np.nonzero(good & ~skip)[0])
    assert 4000 < int((~good & ~skip).sum()) < 10000
    pool = torch.randint(0, 256, (pages, 32), dtype=torch.uint8, generator=g).cuda()
    want = pool.clone()
    want[pairs[done, 1].long().cuda()] = pool[pairs[done, 0].long().cuda()]
    status = i32([0])
    mla.cache_copy_pages(pool, pairs.cuda(), status=status)
    assert torch.equal(pool, want) and int(status) == BAD_INDEX


def test_copy_judges_targets_that_fall_together():
    """Targets at regular distances (the places of a judging table fill unevenly), each once, and read by none."""
    for step in (1, 2, 64, 1024, 2048, 4096):
        n = 3000
        pages = n * step + n
        pairs = torch.stack([torch.arange(n) + n * step, torch.arange(n) * step], 1).int()
        pool = torch.randint(0, 256, (pages, 16), dtype=torch.uint8, device="cuda")
        want = pool.clone()
        want[pairs[:, 1].long().cuda()] = pool[pairs[:, 0].long().cuda()]
        status = i32([0])
        mla.cache_copy_pages(pool, pairs.cuda(), status=status)
        assert torch.equal(pool, want) and int(status) == 0


@pytest.mark.parametrize("length", [-5, 7 * 64 + 1, 2 ** 31 - 1])
def test_compact_reports_a_length_out_of_range(length):
    s = State(3, 200, 40, seed=25)
    s.grow([1], [7 * 64 - s.host.lens[1]])  # a row of all its pages
    s.host.lens[1] = length
    s.lens = i32(s.host.lens)
    s.compact()
    assert s.host.bad


def test_largest_lists_and_tables():
    """65536 rows and lists of 4096 entries, the most that a call takes."""
    rng = random.Random(26)
    s = State(4096, 190, 24000, seed=26, empty_rows=61440, width=4)
    some = rng.sample(range(4096), 4096)
    s.grow(some, [rng.randint(0, 70) if s.host.lens[r] < 186 else 0 for r in some])
    s.fork([rng.randrange(4096) for _ in range(4096)], rng.sample(range(4096, 65536), 4096))
    s.free(rng.sample(range(65536), 4096))
    s.compact()
