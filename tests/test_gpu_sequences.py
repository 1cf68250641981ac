"""Fork, extend and compact on the GPU against the row-by-row restatement of
tests/_sequences_ref.py: equal in every number and byte."""
import random

import pytest
import torch

from tests._sequences_ref import Book, blocks, make_book

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    pa.pa_device_errors(clear=True)
    return pa


def cuda(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class Dev:
    """A Book's tensors on the GPU."""

    def __init__(self, pa, book):
        self.pa, self.bs = pa, book.bs
        self.tables = cuda(book.tables).reshape(len(book.lens), -1)
        self.lens, self.refs = cuda(book.lens), cuda(book.refs)
        self.pools = [p.cuda() for p in book.pools]
        n = pa.pa_sequences_workspace_size(max(1, len(book.lens)), len(book.refs))
        self.ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        self.info = torch.zeros(2, dtype=I32, device="cuda")

    def fork(self, parents, in_place=False):
        out = torch.full((len(parents), self.tables.shape[1]), -9, dtype=I32, device="cuda")
        lens, refs = torch.empty(len(parents), dtype=I32, device="cuda"), self.refs
        if not in_place:
            refs = torch.empty_like(refs)
        before = [t.clone() for t in (self.tables, self.lens, self.refs)]
        self.pa.pa_fork_sequences(out, lens, refs, self.tables, self.lens, self.refs,
                                  cuda(parents), self.bs)
        kept = [self.tables, self.lens] + ([] if in_place else [self.refs])
        assert all(torch.equal(a, b) for a, b in zip(kept, before))
        self.tables, self.lens, self.refs = out, lens, refs

    def extend(self, new, num_slots, in_place=False, stream=None):
        slots = torch.full((num_slots,), -5, dtype=torch.int64, device="cuda")
        to = (self.tables, self.lens, self.refs)
        if not in_place:
            to = (torch.full_like(self.tables, -9), torch.empty_like(self.lens),
                  torch.empty_like(self.refs))
        self.pa.pa_extend_sequences(*to, slots, self.info, self.tables, self.lens, self.refs,
                                    cuda(new), self.pools, self.bs, self.ws, stream=stream)
        self.tables, self.lens, self.refs = to
        return slots.tolist(), self.info.tolist()

    def compact(self, in_place=False):
        ids = torch.full_like(self.refs, -5)
        to = (self.tables, self.refs)
        if not in_place:
            to = torch.full_like(self.tables, -9), torch.full_like(self.refs, -9)
        self.pa.pa_compact_blocks(*to, ids, self.info, self.tables, self.lens, self.refs,
                                  self.pools, self.bs, self.ws)
        self.tables, self.refs = to
        return ids.tolist(), self.info.tolist()

    def same(self, book, flags=0):
        assert self.tables.tolist() == book.tables
        assert self.lens.tolist() == book.lens and self.refs.tolist() == book.refs
        for a, b in zip(self.pools, book.pools):
            assert torch.equal(a.cpu(), b)
        assert self.pa.pa_device_errors(clear=True) == flags


SIZES = [(1, 1, 16, 3), (7, 5, 16, 60), (40, 9, 1, 300), (33, 30, 32, 700), (300, 12, 16, 5000),
         (1100, 3, 7, 2500), (3, 2500, 16, 9000)]


def nines(book, rows=None):
    return [[-9] * len(book.tables[0]) for _ in range(len(book.lens) if rows is None else rows)]


@pytest.mark.parametrize("rows,wide,bs,nb", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(pa, rows, wide, bs, nb, in_place):
    rng = random.Random(rows)
    for out in (rows, max(1, rows // 2), rows + 5):
        book = make_book(rows, wide, bs, nb, seed=rows + out)
        dev = Dev(pa, book)
        for parents in ([rng.randrange(-1, rows) for _ in range(out)], [rng.randrange(rows)] * out):
            parents = [min(p, len(book.lens) - 1) for p in parents]
            book.fork(parents, nines(book, out))
            dev.fork(parents, in_place)
            dev.same(book)


def room_for(book, rng, most):
    wide = len(book.tables[0])
    return [min(rng.choice([0, 1, 1, book.bs, rng.randint(0, most)]), wide * book.bs - n)
            for n in book.lens]


@pytest.mark.parametrize("rows,wide,bs,nb", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(pa, rows, wide, bs, nb, in_place):
    rng = random.Random(rows)
    for seed, share in ((1, 0.0), (2, 0.9), (3, 0.5)):
        book = make_book(rows, wide, bs, nb, seed=seed, share=share, shapes=((2, 3, 32), (1, 7), (3, 4)))
        dev = Dev(pa, book)
        for most in (1, 2 * bs, 40):
            new = room_for(book, rng, most)
            slots = sum(new) + rng.choice([0, 1, 300])
            want = book.extend(new, slots, None if in_place else nines(book))
            assert dev.extend(new, slots, in_place) == want
            dev.same(book, 0 if want[1][1] >= 0 else pa.DEVERR_POOL)


def test_extend_shared_last_blocks(pa):
    """Where all holders of a block go on in it the last keeps it; where one does not,
    all others copy; whole blocks are never copied."""
    bs = 4
    tables = [[0, 1, -7]] * 3 + [[2, -7, -7]] * 3 + [[3, -7, -7]] * 2
    book = Book(tables, [6, 6, 6, 3, 3, 3, 4, 4], [3, 3, 3, 2, 0, 0, 0, 0, 0, 0, 0, 0], bs,
                [torch.arange(24, dtype=torch.int8).view(1, 12, 2)])
    dev = Dev(pa, book)
    new = [1, 1, 1, 1, 0, 2, 1, 1]
    want = book.extend(new, 9)
    assert want[1] == [7, 1]
    assert [r[1] for r in book.tables[:3]] == [4, 5, 1]
    assert dev.extend(new, 9, True) == want
    dev.same(book)


def test_extend_without_room(pa):
    """All or nothing: too few blocks, or a slot_mapping that is too short."""
    book = make_book(6, 20, 16, 40, seed=4)
    free = sum(c == 0 for c in book.refs)
    new = [0] * 6
    new[2] = 20 * 16 - book.lens[2]
    new[3] = 20 * 16 - book.lens[3]
    for slots in (sum(new), sum(new) - 1, 0):
        for in_place in (False, True):
            b = Book(book.tables, book.lens, book.refs, 16, book.pools)
            dev = Dev(pa, b)
            want = b.extend(new, slots, None if in_place else nines(b))
            assert dev.extend(new, slots, in_place) == want
            if want[0] and max(want[0]) >= 0:
                dev.same(b)
            else:
                dev.same(b, pa.DEVERR_POOL)
    assert free < 40


def test_extend_bad_rows(pa):
    """Lengths and numbers outside their ranges count as said, and are flagged."""
    book = make_book(5, 4, 16, 60, seed=6, share=0)
    dev = Dev(pa, book)
    new = [1, -3, 1, 1, 4 * 16 + 1]
    ok = [n if 0 <= n <= 64 - have else 0 for n, have in zip(new, book.lens)]
    want = book.extend(ok, 10)
    assert dev.extend(new, 10, True) == want
    dev.same(book, pa.DEVERR_SEQ_LEN)
    dev.lens[0], dev.lens[1] = -1, 4 * 16 + 5
    dev.extend([0] * 5, 4, True)
    assert dev.lens.tolist()[:2] == [0, 64]
    assert pa.pa_device_errors(clear=True) & pa.DEVERR_SEQ_LEN


def test_bad_ids_are_flagged(pa):
    book = make_book(4, 4, 16, 40, seed=7, share=0)
    book.lens[1] = 17
    for bad in (-3, 40, 1 << 30):
        dev = Dev(pa, book)
        dev.tables[1, 0], dev.tables[1, 1] = bad, bad
        dev.fork([1, 1, -1, 3])
        assert dev.tables[0, 0].item() == bad
        assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID
        slots, _ = dev.extend([1, 0, 0, 0], 1)
        assert slots == [-1]
        assert pa.pa_device_errors(clear=True) & pa.DEVERR_BLOCK_ID
        dev.compact()
        assert dev.tables[1, 0].item() == -1
        assert pa.pa_device_errors(clear=True) & pa.DEVERR_BLOCK_ID
    dev = Dev(pa, make_book(4, 4, 16, 40, seed=7, share=0))
    dev.fork([4, -5, 1 << 30])
    assert dev.lens.tolist() == [0, 0, 0]
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_PARENT


@pytest.mark.parametrize("rows,wide,bs,nb", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(pa, rows, wide, bs, nb, in_place):
    for seed in (1, 2):
        book = make_book(rows, wide, bs, nb, seed=seed, shapes=((2, 3, 32), (1, 7), (2, 48)))
        keep = random.Random(seed)
        book.fork([r if keep.random() < 0.6 else -1 for r in range(rows)], book.tables)
        dev = Dev(pa, book)
        for _ in range(2):                 # the second time nothing moves
            want = book.compact(None if in_place else nines(book))
            assert dev.compact(in_place) == want
            dev.same(book)
        assert want[1][1] == 0


def test_compact_ends(pa):
    """Nothing in use, everything in use, and all of it at the end."""
    for refs in ([0] * 5000, [2] * 5000, [0] * 4000 + [1] * 1000, [1] * 1000 + [0] * 4000,
                 [0, 1] * 2500, [0]):
        pool = torch.arange(len(refs)).to(torch.int8).view(1, -1, 1)
        book = Book([[-1]], [0], refs, 16, [pool])
        dev = Dev(pa, book)
        want = book.compact(nines(book))
        assert dev.compact() == want
        dev.same(book)


def test_many_pools_of_every_alignment(pa):
    """More pools than a small parameter block holds, bytes of odd sizes, offsets of
    one byte and of four, blocks of more than one unit."""
    book = make_book(9, 6, 4, 80, seed=9, share=0.8)
    g = torch.Generator().manual_seed(1)
    sizes = [1, 2, 3, 4, 12, 16, 20, 48, 16384, 16388, 40000, 65537] * 2
    book.pools = [torch.randint(0, 100, (1 + i % 3, 80, n), generator=g, dtype=torch.int8)
                  for i, n in enumerate(sizes)]
    dev = Dev(pa, book)
    for i, p in enumerate(dev.pools):      # some begin off 16 bytes
        off = (0, 1, 4, 16)[i % 4]
        room = torch.zeros(p.numel() + 16, dtype=torch.int8, device="cuda")
        dev.pools[i] = room[off:off + p.numel()].view(p.shape).copy_(p)
    new = [min(1, 24 - n) for n in book.lens]
    assert dev.extend(new, 9) == book.extend(new, 9, nines(book))
    dev.same(book)
    book.fork([0, 1, 2, -1, -1, 5, -1, 7, 8], nines(book))
    dev.fork([0, 1, 2, -1, -1, 5, -1, 7, 8])
    assert dev.compact() == book.compact(nines(book))
    dev.same(book)


def test_far_blocks(pa):
    """Blocks that begin past 2^32 bytes of their plane."""
    nb, size = 70000, 65536                # 4.6 GB a plane
    pool = torch.zeros(1, nb, size, dtype=torch.int8, device="cuda")
    pool[0, nb - 1] = 5
    pool[0, nb - 2] = 6
    refs = torch.zeros(nb, dtype=I32, device="cuda")
    refs[nb - 2:] = cuda([1, 2])
    tables = cuda([[nb - 1, nb - 2], [nb - 1, -1]])
    lens = cuda([24, 10])
    ws = torch.empty(pa.pa_sequences_workspace_size(2, nb), dtype=torch.uint8, device="cuda")
    info, ids = torch.zeros(2, dtype=I32, device="cuda"), torch.empty_like(refs)
    slots = torch.empty(2, dtype=torch.int64, device="cuda")
    pa.pa_extend_sequences(tables, lens, refs, slots, info, tables, lens, refs, cuda([0, 1]), [pool],
                           16, ws)         # row 1 copies its shared last block to block 0
    assert tables.tolist() == [[nb - 1, nb - 2], [0, -1]] and slots.tolist() == [10, -1]
    assert bool((pool[0, 0] == 5).all()) and not pool[0, 1].any()
    pa.pa_compact_blocks(tables, refs, ids, info, tables, lens, refs, [pool], 16, ws)
    assert tables.tolist() == [[2, 1], [0, -1]] and info.tolist() == [3, 2]
    assert bool((pool[0, 1] == 6).all()) and bool((pool[0, 2] == 5).all())
    assert pa.pa_device_errors(clear=True) == 0


def test_capture_and_replay(pa):
    """A step captured once: fork, extend and compact follow whatever the tensors hold
    at the time of the replay."""
    book = make_book(8, 10, 16, 200, seed=11)
    dev = Dev(pa, book)
    parents, new = cuda([0] * 8), cuda([1] * 8)
    t = [[torch.full_like(dev.tables, -9), torch.empty_like(dev.lens), torch.empty_like(dev.refs)]
         for _ in range(3)]
    slots, ids = torch.empty(80, dtype=torch.int64, device="cuda"), torch.empty_like(dev.refs)

    def step():
        pa.pa_fork_sequences(*t[0], dev.tables, dev.lens, dev.refs, parents, 16)
        pa.pa_extend_sequences(*t[1], slots, dev.info, *t[0], new, dev.pools, 16, dev.ws)
        pa.pa_compact_blocks(t[2][0], t[2][2], ids, dev.info, *t[1], dev.pools, 16, dev.ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = random.Random(5)
    for seed in range(4):
        book = make_book(8, 10, 16, 200, seed=20 + seed)
        dev.tables.copy_(cuda(book.tables))
        dev.lens.copy_(cuda(book.lens))
        dev.refs.copy_(cuda(book.refs))
        for a, b in zip(dev.pools, book.pools):
            a.copy_(b)
        for x in t:
            x[0].fill_(-9)
        par = [rng.randrange(-1, 8) for _ in range(8)]
        parents.copy_(cuda(par))
        book.fork(par, nines(book))
        n = room_for(book, rng, 20)
        new.copy_(cuda(n))
        g.replay()
        want, _ = book.extend(n, 80, nines(book))
        wids, winfo = book.compact(nines(book))
        assert slots.tolist() == want and ids.tolist() == wids and dev.info.tolist() == winfo
        assert t[2][0].tolist() == book.tables and t[2][2].tolist() == book.refs
        for a, b in zip(dev.pools, book.pools):
            assert torch.equal(a.cpu(), b)
    assert pa.pa_device_errors(clear=True) == 0


def test_no_rows(pa):
    refs, out = cuda([0, 3, 0]), torch.empty(3, dtype=I32, device="cuda")
    none, lens = torch.empty(0, 4, dtype=I32, device="cuda"), torch.empty(0, dtype=I32, device="cuda")
    info, slots = cuda([9, 9]), cuda([5, 5], torch.int64)
    ws = torch.empty(pa.pa_sequences_workspace_size(0, 3), dtype=torch.uint8, device="cuda")
    pa.pa_fork_sequences(none, lens, out, none, lens, refs, lens, 16)
    assert out.tolist() == [0, 3, 0]
    pa.pa_extend_sequences(none, lens, out, slots, info, none, lens, refs, lens, [], 16, ws)
    assert info.tolist() == [0, 2] and slots.tolist() == [-1, -1]
    ids = torch.empty_like(refs)
    pa.pa_compact_blocks(none, out, ids, info, none, lens, refs, [], 16, ws)
    assert ids.tolist() == [-1, 0, -1] and out.tolist() == [3, 0, 0] and info.tolist() == [1, 1]
    assert pa.pa_device_errors(clear=True) == 0


def test_two_streams(pa):
    """Two programs' steps at once, a workspace each."""
    books = [make_book(50, 12, 16, 900, seed=s, share=0.7) for s in (1, 2)]
    devs = [Dev(pa, b) for b in books]
    rng = random.Random(1)
    news = [room_for(b, rng, 30) for b in books]
    streams = [torch.cuda.Stream() for _ in books]
    torch.cuda.synchronize()
    got = []
    for d, n, s in zip(devs, news, streams):
        with torch.cuda.stream(s):
            got.append(d.extend(n, sum(n), True))
    for d, b, n, g in zip(devs, books, news, got):
        assert g == b.extend(n, sum(n))
        d.same(b)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", [-3, 40, 1 << 30])
def test_extend_flags_ids_in_any_entry(pa, bad, in_place):
    """An id outside the pool anywhere in a row, whether the row grows or not; entries
    behind a row's last are not looked at."""
    book = Book([[3, 5, 7, -7], [9, 11, bad, bad], [2, bad, bad, bad]], [40, 20, 0],
                [int(b in (3, 5, 7, 9, 11)) for b in range(40)], 16)
    for row, new in ((0, [1, 0, 0]), (0, [0, 0, 0]), (1, [0, 1, 3])):
        dev = Dev(pa, book)
        dev.extend(new, 4, in_place)
        assert pa.pa_device_errors(clear=True) == 0
        dev = Dev(pa, book)
        dev.tables[row, 0] = bad
        dev.extend(new, 4, in_place)
        assert dev.tables[row, 0].item() == bad
        assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_in_a_free_block(pa, in_place):
    """A last block of count 0 is handed to whoever needs one: no token of the row that
    still names it goes there."""
    book = Book([[0, -7, -7], [1, -7, -7], [-7, -7, -7]], [10, 10, 0], [0, 1, 0, 0, 0], 16)
    dev = Dev(pa, book)
    slots, info = dev.extend([8, 2, 3], 13, in_place)
    assert info == [2, 2]
    # row 0's second block and row 2's first are the lowest free ones, 0 and 2
    assert slots == [-1] * 6 + [0, 1, 26, 27, 32, 33, 34]
    assert dev.refs.tolist() == [1, 1, 1, 0, 0] and dev.lens.tolist() == [18, 12, 3]
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID
