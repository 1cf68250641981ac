"""Selection of blocks, and decode over an e4m3 pool with block scales and over
listed blocks, against their 64-bit restatement."""
import math

import pytest
import torch

from tests import _block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    pa.pa_device_errors(clear=True)
    return pa


def _workspace(pa, h, hkv, d):
    ws = torch.empty(pa.pa_block_decode_workspace_size(h, hkv, d), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                       # NaN: its contents on entry do not matter
    return ws


def _inputs(lens, h, hkv, d, bs, dtype, eight, seed=1, spread=1.0, width=0):
    tables, nb = R.make_tables(lens, bs, seed=seed, width=width)
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, eight, seed=seed, spread=spread)
    R.poison_tails(pool, tables, lens, bs)
    q = torch.randn(len(lens), h, d, generator=R.gen(seed + 1, "cuda"), device="cuda").to(dtype)
    return q, pool, scales, tables, R.ints(lens)


def _check(pa, got, lse, ref, dtype, eight):
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    R.check_decode(got, ref, half_products=eight or dtype == torch.float16,
                   two_parts=not (eight and dtype == torch.bfloat16), lse=lse)


HEADS = [(4, 4), (8, 1), (16, 8), (12, 3), (32, 32), (10, 5), (64, 8), (24, 12), (14, 7), (11, 11),
         (36, 9)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("h,hkv", HEADS)
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
def test_decode_fp8_block(pa, d, bs, h, hkv, dtype):
    lens = [1, 0, 15, 16, 17, 300, 33, 1025]
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, dtype, True)
    out, lse = torch.full_like(q, math.nan), torch.empty(q.shape[:2], device="cuda")
    scale = 1 / math.sqrt(d)
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, scale, bs, max(lens),
                           _workspace(pa, h, hkv, d), lse=lse)
    assert torch.count_nonzero(out[1]) == 0
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, scale), dtype, True)


@pytest.mark.parametrize("h,hkv,d,bs", [(8, 1, 128, 16), (64, 8, 128, 32), (4, 4, 64, 16),
                                        (24, 3, 128, 16), (5, 5, 64, 32), (14, 7, 128, 32)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_fp8_block_long(pa, h, hkv, d, bs, dtype):
    """Cut over many CTAs, beside short sequences; a group of few heads."""
    lens = [20011, 3, 700]
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, dtype, True, seed=7)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.11, bs, max(lens),
                           _workspace(pa, h, hkv, d), lse=lse)
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, 0.11), dtype, True)


def test_decode_fp8_block_many_sequences(pa):
    """More sequences than threads of a CTA, most of one token."""
    lens = [1 + (i * 37) % 5 for i in range(700)]
    lens[333] = 500
    q, pool, scales, tables, sl = _inputs(lens, 4, 2, 64, 16, torch.float16, True, seed=11)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.125, 16, 500,
                           _workspace(pa, 4, 2, 64), lse=lse)
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, 16, 0.125), torch.float16, True)


def test_decode_fp8_block_extreme_scales(pa):
    """Value scales over 2^-40 .. 2^40 within one row: the small blocks' weight
    still counts in the normaliser, the large blocks' values in the output."""
    lens, h, hkv, d, bs = [256, 90], 8, 2, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.bfloat16, True, spread=0.0)
    scales[1] *= torch.exp2(torch.randint(-40, 41, scales[1].shape, generator=R.gen(2, "cuda"),
                                          device="cuda").float())
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.1, bs, 256,
                           _workspace(pa, h, hkv, d), lse=lse)
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, 0.1), torch.bfloat16, True)


def test_decode_fp8_block_peaked_rows(pa):
    """Large queries: nearly one-hot softmaxes, some of them on the last token."""
    lens, h, hkv, d, bs = [513, 40, 2], 8, 2, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True)
    q *= 30
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.09, bs, 600,
                           _workspace(pa, h, hkv, d), lse=lse)
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, 0.09), torch.float16, True)


def test_decode_flags(pa):
    lens, h, hkv, d, bs = [40, 64, 50], 8, 2, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True)
    ws, out = _workspace(pa, h, hkv, d), torch.empty_like(q)
    bad = tables.clone()
    bad[0, 1] = 10 ** 6                              # reads as zeros
    pa.pa_decode_fp8_block(out, q, pool, scales, bad, sl, 0.1, bs, 64, ws)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID
    R.check_decode(out, R.ref_decode(q, pool, scales, bad, sl, bs, 0.1), True, True)
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, R.ints([40, 65, -3]), 0.1, bs, 64, ws)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    R.check_decode(out, R.ref_decode(q, pool, scales, tables, R.ints([40, 64, 0]), bs, 0.1), True,
                   True)


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------
def _bounds(pa, pool, scales, tables, lens, bs, hkv, d):
    nb = pool.shape[1]
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.ones(nb, hkv, device="cuda")
    pa.pa_update_block_bounds(bounds, bsc, pool, tables, R.ints(lens), R.starts(lens), bs,
                              max(lens), kv_scales=scales)
    return bounds, bsc


def _select(pa, q, bounds, bsc, tables, sl, bs, most, sink, recent, msl):
    b, hkv = q.shape[0], bounds.shape[1]
    lists = torch.full((b, hkv, most), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_select_blocks_workspace_size(b, hkv, msl, bs), dtype=torch.uint8,
                     device="cuda")
    pa.pa_select_blocks(lists, counts, q, bounds, bsc, tables, sl, bs, msl, ws,
                        num_sink_blocks=sink, num_recent_blocks=recent)
    return lists, counts


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("h,hkv,d,bs,most,sink,recent", [
    (8, 8, 128, 16, 5, 1, 1), (8, 1, 64, 16, 16, 0, 0), (64, 8, 128, 32, 9, 2, 3),
    (12, 3, 64, 32, 1, 0, 1), (6, 3, 128, 16, 64, 64, 0), (10, 5, 128, 16, 33, 0, 33)])
def test_select(pa, h, hkv, d, bs, most, sink, recent, dtype):
    lens = [1, 0, bs * most, bs * most + 1, 2500, 1000, 77]
    q, pool, _, tables, sl = _inputs(lens, h, hkv, d, bs, dtype, False, seed=21)
    bounds, bsc = _bounds(pa, pool, None, tables, lens, bs, hkv, d)
    got = _select(pa, q, bounds, bsc, tables, sl, bs, most, sink, recent, max(lens))
    want = R.ref_select(q, bounds, bsc, tables, sl, bs, most, sink, recent)
    assert pa.pa_device_errors(clear=True) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_select_ties_take_the_lowest_position(pa):
    """Identical bounds everywhere, and a few better blocks."""
    h, hkv, d, bs, n = 4, 2, 128, 16, 3000
    tables, nb = R.make_tables([n * bs], bs)
    bounds = torch.full((nb, hkv, 2, d), 3, dtype=torch.int8, device="cuda")
    bsc = torch.ones(nb, hkv, device="cuda")
    q = torch.ones(1, h, d, dtype=torch.float16, device="cuda")
    for j in (2999, 1500, 7):
        bounds[tables[0, j], 1] = 4
    sl = R.ints([n * bs])
    lists, counts = _select(pa, q, bounds, bsc, tables, sl, bs, 10, 0, 0, n * bs)
    assert counts.tolist() == [10]
    assert lists[0, 0].tolist() == list(range(10))
    assert lists[0, 1].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 1500, 2999]


def test_select_odd_values(pa):
    """Queries with NaN, infinities, zeros and tiny values; blocks whose scale is
    infinite; negative scores; scales far apart."""
    h, hkv, d, bs, n = 8, 2, 64, 16, 200
    tables, nb = R.make_tables([n * bs] * 3, bs, seed=2)
    g = R.gen(3, "cuda")
    bounds = torch.randint(-127, 128, (nb, hkv, 2, d), generator=g, device="cuda")
    bounds = bounds.sort(2, descending=True).values.to(torch.int8)
    bsc = torch.exp2(torch.randint(-60, 61, (nb, hkv), generator=g, device="cuda").float())
    bsc[tables[0, 150], 1] = math.inf
    bounds[tables[0, 150], 1] = 0
    q = torch.randn(3, h, d, generator=g, device="cuda").to(torch.bfloat16)
    q[0, 0, 3] = math.nan
    q[0, 5, 0], q[0, 5, 1] = math.inf, -math.inf
    q[1, :4] = 0.0
    q[1, 4:] = -1e-30
    sl = R.ints([n * bs, n * bs - 5, 17 * bs])
    got = _select(pa, q, bounds, bsc, tables, sl, bs, 24, 1, 1, n * bs)
    want = R.ref_select(q, bounds, bsc, tables, sl, bs, 24, 1, 1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert 150 in got[0][0, 1].tolist()


@pytest.mark.parametrize("b,h,hkv,n,most", [
    (1, 2, 1, 5000, 200),      # one CTA cluster, keys in two rounds
    (40, 32, 8, 90, 7),        # more (sequence, head)s than CTAs fit: eight heads a cluster
    (10, 16, 8, 333, 64), (3, 24, 12, 150, 31), (2, 4, 4, 70000, 100)])
def test_select_shapes_of_the_grid(pa, b, h, hkv, n, most):
    """Small codes, so that scores tie often, also at the border."""
    d, bs, g = 64, 16, R.gen(b, "cuda")
    lens = [bs * n - 3 * i for i in range(b)]
    tables, nb = R.make_tables(lens, bs, seed=b)
    up = torch.randint(0, 4, (nb, hkv, 1, d), generator=g, device="cuda")
    bounds = torch.cat((up, up - 1), 2).to(torch.int8)
    bsc = torch.exp2(torch.randint(-1, 2, (nb, hkv), generator=g, device="cuda").float())
    q = torch.randn(b, h, d, generator=g, device="cuda").to(torch.bfloat16)
    got = _select(pa, q, bounds, bsc, tables, R.ints(lens), bs, most, 1, 2, max(lens))
    want = R.ref_select(q, bounds, bsc, tables, R.ints(lens), bs, most, 1, 2)
    assert pa.pa_device_errors(clear=True) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_select_many_blocks(pa):
    h, hkv, d, bs = 16, 2, 64, 16
    lens = [16 * 20000, 5000]
    tables, nb = R.make_tables(lens, bs, seed=4)
    g = R.gen(5, "cuda")
    # few distinct codes: many ties at the border
    bounds = torch.randint(0, 2, (nb, hkv, 2, d), generator=g, device="cuda").to(torch.int8)
    bsc = torch.ones(nb, hkv, device="cuda")
    q = torch.ones(2, h, d, device="cuda", dtype=torch.float16)
    got = _select(pa, q, bounds, bsc, tables, R.ints(lens), bs, 300, 2, 2, max(lens))
    want = R.ref_select(q, bounds, bsc, tables, R.ints(lens), bs, 300, 2, 2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_select_flags(pa):
    lens, h, hkv, d, bs = [320, 320], 4, 2, 128, 16
    q, pool, _, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, False)
    bounds, bsc = _bounds(pa, pool, None, tables, lens, bs, hkv, d)
    bad = tables.clone()
    bad[0, 4] = -1
    _select(pa, q, bounds, bsc, bad, sl, bs, 3, 0, 1, 320)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID
    lists, counts = _select(pa, q, bounds, bsc, tables, R.ints([-4, 9999]), bs, 3, 0, 1, 320)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    assert counts.tolist() == [0, 3] and (lists[0] == -1).all()


# ---------------------------------------------------------------------------
# Sparse decode
# ---------------------------------------------------------------------------
def _random_lists(lens, hkv, most, bs, seed, shuffle=True):
    g = R.gen(seed, "cpu")
    lists = torch.full((len(lens), hkv, most), -1, dtype=torch.int32)
    counts = []
    for s, length in enumerate(lens):
        n = -(-length // bs)
        counts.append(min(n, most))
        for k in range(hkv):
            pick = torch.randperm(n, generator=g)[:counts[-1]]
            lists[s, k, :counts[-1]] = (pick if shuffle else pick.sort().values).int()
    return lists.cuda(), R.ints(counts)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("h,hkv,d,bs,most", [
    (4, 4, 64, 16, 7), (8, 1, 128, 16, 64), (64, 8, 128, 32, 20), (12, 3, 64, 32, 5),
    (32, 32, 128, 16, 1), (10, 5, 128, 32, 40), (7, 7, 64, 16, 3), (12, 6, 128, 16, 12)])
def test_sparse(pa, h, hkv, d, bs, most, dtype, eight):
    lens = [1, 0, 500, 17, 2000, 31]
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, dtype, eight, seed=31)
    lists, counts = _random_lists(lens, hkv, most, bs, 5)
    out, lse = torch.full_like(q, math.nan), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_sparse(out, q, pool, tables, sl, lists, counts, 0.12, bs,
                        _workspace(pa, h, hkv, d), kv_scales=scales, lse=lse)
    assert torch.count_nonzero(out[1]) == 0
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, 0.12, lists, counts), dtype,
           eight)


@pytest.mark.parametrize("eight", [False, True])
def test_sparse_padding_repeats_and_empty_lists(pa, eight):
    lens, h, hkv, d, bs = [200, 200, 200, 200], 8, 2, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, eight)
    lists = torch.full((4, hkv, 6), 10 ** 6, dtype=torch.int32, device="cuda")  # never read
    counts = R.ints([6, 4, 0, 5])
    lists[0, 0] = R.ints([-1, 3, -1, 3, 12, -5])       # padding; block 3 twice; the last block
    lists[0, 1] = R.ints([-1] * 6)                     # a head with no block at all
    lists[1, 0, :4] = R.ints([12, 0, 5, 7])
    lists[1, 1, :4] = R.ints([0, 1, 2, 3])
    lists[3, :, :5] = R.ints([4, 9, 1, 2, 11])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pa.pa_decode_sparse(out, q, pool, tables, sl, lists, counts, 0.1, bs,
                        _workspace(pa, h, hkv, d), kv_scales=scales, lse=lse)
    assert torch.count_nonzero(out[0, 4:]) == 0 and torch.count_nonzero(out[2]) == 0
    _check(pa, out, lse, R.ref_decode(q, pool, scales, tables, sl, bs, 0.1, lists, counts),
           torch.float16, eight)


def test_sparse_flags(pa):
    lens, h, hkv, d, bs = [64, 64], 4, 2, 64, 16
    q, pool, _, tables, sl = _inputs(lens, h, hkv, d, bs, torch.bfloat16, False)
    lists, counts = _random_lists(lens, hkv, 3, bs, 1)
    ws, out = _workspace(pa, h, hkv, d), torch.empty_like(q)
    past = lists.clone()
    past[0, 1, 2] = 4                                   # the sequence has blocks 0..3
    pa.pa_decode_sparse(out, q, pool, tables, sl, past, counts, 0.1, bs, ws)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_BLOCK_ID
    R.check_decode(out, R.ref_decode(q, pool, None, tables, sl, bs, 0.1, past, counts), False, True)
    pa.pa_decode_sparse(out, q, pool, tables, sl, lists, R.ints([9, -1]), 0.1, bs, ws)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    R.check_decode(out, R.ref_decode(q, pool, None, tables, sl, bs, 0.1, lists, R.ints([3, 0])),
                   False, True)


def test_sparse_over_every_block_is_decode(pa):
    """All blocks listed in order: the dense call's result, bit for bit."""
    lens, h, hkv, d, bs = [700, 33, 1], 16, 4, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True)
    n = -(-700 // bs)
    lists = torch.arange(n, dtype=torch.int32, device="cuda").expand(3, hkv, n).contiguous()
    counts = R.ints([-(-v // bs) for v in lens])
    ws, a, b = _workspace(pa, h, hkv, d), torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_fp8_block(a, q, pool, scales, tables, sl, 0.1, bs, 700, ws)
    pa.pa_decode_sparse(b, q, pool, tables, sl, lists, counts, 0.1, bs, ws, kv_scales=scales)
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
class _Server:
    """A small serving loop over one e4m3 pool: prompts, then steps of write,
    bounds, selection and sparse decode."""

    def __init__(self, pa, dtype=torch.bfloat16, h=16, hkv=4, d=128, bs=16, most=6):
        self.pa, self.h, self.hkv, self.d, self.bs, self.most = pa, h, hkv, d, bs, most
        self.lens, self.room = [130, 7, 256], 300
        self.tables, self.nb = R.make_tables([self.room] * 3, bs, seed=8)
        self.pool = torch.full((2, self.nb, bs, hkv, d), 0x7F, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((2, self.nb, hkv), math.nan, device="cuda")
        self.bounds = torch.zeros(self.nb, hkv, 2, d, dtype=torch.int8, device="cuda")
        self.bsc = torch.zeros(self.nb, hkv, device="cuda")
        self.lists = torch.zeros(3, hkv, most, dtype=torch.int32, device="cuda")
        self.counts = torch.zeros(3, dtype=torch.int32, device="cuda")
        self.sl = R.ints(self.lens)
        self.ones = R.starts([1, 1, 1])
        self.g, self.dtype = R.gen(12, "cuda"), dtype
        self.ws = _workspace(pa, h, hkv, d)
        self.sws = torch.empty(pa.pa_select_blocks_workspace_size(3, hkv, self.room, bs),
                               dtype=torch.uint8, device="cuda")
        self.q, self.k, self.v = (self.rand(3, x) for x in (h, hkv, hkv))
        self.out = torch.empty_like(self.q)
        n = sum(self.lens)
        self.append(self.rand(n, hkv), self.rand(n, hkv), R.starts(self.lens), max(self.lens))

    def rand(self, n, heads):
        return torch.randn(n, heads, self.d, generator=self.g, device="cuda").to(self.dtype)

    def append(self, k, v, qsl, most):
        self.pa.pa_reshape_and_cache_fp8_block(k, v, self.pool, self.scales, self.tables, self.sl,
                                               qsl, self.bs, most)
        self.pa.pa_update_block_bounds(self.bounds, self.bsc, self.pool, self.tables, self.sl, qsl,
                                       self.bs, most, kv_scales=self.scales)

    def step(self):
        self.append(self.k, self.v, self.ones, 1)
        self.pa.pa_select_blocks(self.lists, self.counts, self.q, self.bounds, self.bsc,
                                 self.tables, self.sl, self.bs, self.room, self.sws,
                                 num_sink_blocks=1, num_recent_blocks=1)
        self.pa.pa_decode_sparse(self.out, self.q, self.pool, self.tables, self.sl, self.lists,
                                 self.counts, 0.09, self.bs, self.ws, kv_scales=self.scales)

    def next_inputs(self):
        self.lens = [v + 1 for v in self.lens]
        self.sl.copy_(R.ints(self.lens))
        for t, x in ((self.q, self.h), (self.k, self.hkv), (self.v, self.hkv)):
            t.copy_(self.rand(3, x))

    def expect(self, pool, scales, bounds, bsc):
        """The step's results from the state before it, in 64 bits."""
        pool, scales = R.ref_write(self.k, self.v, pool, scales, self.tables, self.sl, self.ones,
                                   self.bs)
        bounds, bsc = R.ref_bounds(bounds, bsc, pool, scales, self.tables, self.sl, self.ones,
                                   self.bs)
        lists, counts = R.ref_select(self.q, bounds, bsc, self.tables, self.sl, self.bs, self.most,
                                     1, 1)
        ref = R.ref_decode(self.q, pool, scales, self.tables, self.sl, self.bs, 0.09, lists, counts)
        return pool, scales, bounds, bsc, lists, counts, ref

    def check(self, want):
        for got, ref in zip((self.pool, self.bounds, self.lists, self.counts),
                            (want[0], want[2], want[4], want[5])):
            assert torch.equal(got, ref)
        for got, ref in ((self.scales, want[1]), (self.bsc, want[3])):
            assert torch.equal(got.nan_to_num(-1.0), ref.nan_to_num(-1.0))
        R.check_decode(self.out, want[6], True, self.dtype == torch.float16)

    def state(self):
        return tuple(t.clone() for t in (self.pool, self.scales, self.bounds, self.bsc))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_serving_steps(pa, dtype):
    s = _Server(pa, dtype)
    for _ in range(20):                                 # past the end of blocks
        s.next_inputs()
        want = s.expect(*s.state())
        s.step()
        s.check(want)
    assert pa.pa_device_errors(clear=True) == 0


def test_serving_steps_in_a_graph(pa):
    """The step captured once and replayed on new inputs, lengths included, on a
    stream of its own."""
    s = _Server(pa)
    s.next_inputs()
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    side = torch.cuda.Stream()
    for _ in range(4):
        s.next_inputs()
        want = s.expect(*s.state())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        s.check(want)
    assert pa.pa_device_errors(clear=True) == 0


def test_two_graphs_share_a_workspace(pa):
    """Captured apart, replayed in turn: each leaves nothing that the other sees."""
    runs, ws = [], _workspace(pa, 16, 2, 128)
    for i, lens in enumerate(([5000, 70], [33, 2500, 900, 1])):
        q, pool, scales, tables, sl = _inputs(lens, 16, 2, 128, 16, torch.float16, True, seed=60 + i)
        out = torch.empty_like(q)
        args = (out, q, pool, scales, tables, sl, 0.1, 16, max(lens), ws)
        pa.pa_decode_fp8_block(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_decode_fp8_block(*args)
        runs.append((graph, out, R.ref_decode(q, pool, scales, tables, sl, 16, 0.1), args))
    for graph, out, ref, _ in (runs[0], runs[1], runs[0], runs[0], runs[1]):
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        R.check_decode(out, ref, True, True)


def test_offsets_beyond_32_bits(pa):
    """A pool of 6 GB: the blocks in use lie in its last part, whose byte offsets
    pass 2^31 in a plane; every operator on them."""
    h, hkv, d, bs, lens = 16, 8, 128, 16, [200, 40]
    nb = 190_000
    tables, used = R.make_tables(lens, bs, extra=0)
    tables = torch.where(tables >= 0, tables + nb - used, -1).int()
    pool = torch.zeros(2, nb, bs, hkv, d, dtype=torch.uint8, device="cuda")
    scales = torch.ones(2, nb, hkv, device="cuda")
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.ones(nb, hkv, device="cuda")
    g, sl, qsl = R.gen(1, "cuda"), R.ints(lens), R.starts(lens)
    k, v = (torch.randn(sum(lens), hkv, d, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(2, h, d, generator=g, device="cuda").half()
    pa.pa_reshape_and_cache_fp8_block(k, v, pool, scales, tables, sl, qsl, bs, max(lens))
    pa.pa_update_block_bounds(bounds, bsc, pool, tables, sl, qsl, bs, max(lens), kv_scales=scales)
    lists, counts = _select(pa, q, bounds, bsc, tables, sl, bs, 5, 1, 1, 200)
    ws, out, sparse = _workspace(pa, h, hkv, d), torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.1, bs, 200, ws)
    pa.pa_decode_sparse(sparse, q, pool, tables, sl, lists, counts, 0.1, bs, ws, kv_scales=scales)
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    assert not pool[:, :nb - used].any()
    # the same on a pool of the used blocks alone
    near = torch.where(tables >= 0, tables - (nb - used), -1).int()
    tail = slice(nb - used, nb)
    zero = torch.zeros(2, used, bs, hkv, d, dtype=torch.uint8, device="cuda")
    want = R.ref_write(k, v, zero, torch.ones(2, used, hkv, device="cuda"), near, sl, qsl, bs)
    assert torch.equal(pool[:, tail], want[0]) and torch.equal(scales[:, tail], want[1])
    wb = R.ref_bounds(bounds[tail], bsc[tail], *want, near, sl, qsl, bs)
    assert torch.equal(bounds[tail], wb[0]) and torch.equal(bsc[tail], wb[1])
    wl = R.ref_select(q, *wb, near, sl, bs, 5, 1, 1)
    assert torch.equal(lists, wl[0]) and torch.equal(counts, wl[1])
    R.check_decode(out, R.ref_decode(q, *want, near, sl, bs, 0.1), True, True)
    R.check_decode(sparse, R.ref_decode(q, *want, near, sl, bs, 0.1, lists, counts), True, True)


def test_decode_of_not_finite_values(pa):
    """A NaN key or value in the cache reaches its rows and no others; what lies
    behind the last token does not."""
    lens, h, hkv, d, bs = [50, 50, 50], 4, 2, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True)
    ref = R.ref_decode(q, pool, scales, tables, sl, bs, 0.1)
    pool[0, tables[0, 1], 3, 0, 5] = 0x7F              # a key of head 0
    pool[1, tables[2, 3], 1, 1, 7] = 0xFF              # a value of head 1: token 49
    out = torch.empty_like(q)
    pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.1, bs, 50, _workspace(pa, h, hkv, d))
    assert torch.isnan(out[0, :2]).all() and torch.isnan(out[2, 2:, 7]).all()
    assert torch.isnan(out).sum() == 2 * d + 2
    fine = ~torch.isnan(out)
    part = tuple(torch.where(fine, x, 0.0) if x.dim() == 3 else x for x in ref)
    R.check_decode(torch.where(fine, out, 0.0), part, True, True)


def test_two_streams_with_their_own_workspaces(pa):
    """Decodes of different problems in flight at once on two streams."""
    runs = []
    for i, (lens, h, hkv, d, bs) in enumerate((([3000, 50], 16, 2, 128, 16),
                                               ([900, 1200, 4], 8, 8, 64, 32))):
        q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True, seed=40 + i)
        ref = R.ref_decode(q, pool, scales, tables, sl, bs, 0.1)
        runs.append((q, pool, scales, tables, sl, bs, max(lens), _workspace(pa, h, hkv, d), ref,
                     torch.cuda.Stream(), torch.empty_like(q)))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, pool, scales, tables, sl, bs, msl, ws, ref, st, out in runs:
            pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.1, bs, msl, ws, stream=st)
    torch.cuda.synchronize()
    for q, pool, scales, tables, sl, bs, msl, ws, ref, st, out in runs:
        R.check_decode(out, ref, True, True)


def test_results_do_not_change_from_call_to_call(pa):
    lens, h, hkv, d, bs = [9000, 31, 500], 8, 1, 128, 16
    q, pool, scales, tables, sl = _inputs(lens, h, hkv, d, bs, torch.float16, True)
    ws, first = _workspace(pa, h, hkv, d), torch.empty_like(q)
    pa.pa_decode_fp8_block(first, q, pool, scales, tables, sl, 0.1, bs, 9000, ws)
    for _ in range(5):
        out = torch.empty_like(q)
        pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.1, bs, 9000, ws)
        assert torch.equal(out, first)
