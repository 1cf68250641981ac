"""pa_select_blocks where little is left to choose by score, or the bounds are
at the ends of their range: the lists against what the definition gives."""
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


GUARD = 64  # entries before and behind the lists that no call may touch


def _select(pa, q, bounds, bsc, tables, sl, bs, most, sink, recent):
    b, hkv = q.shape[0], bounds.shape[1]
    msl = tables.shape[1] * bs
    n = b * hkv * most
    room = torch.full((n + 2 * GUARD,), -7, dtype=torch.int32, device="cuda")
    lists = room[GUARD:GUARD + n].view(b, hkv, most)
    counts = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((pa.pa_select_blocks_workspace_size(b, hkv, msl, bs),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    pa.pa_select_blocks(lists, counts, q, bounds, bsc, tables, sl, bs, msl, ws,
                        num_sink_blocks=sink, num_recent_blocks=recent)
    assert (room[:GUARD] == -7).all() and (room[GUARD + n:] == -7).all()
    return lists, counts


# (sequences, heads, kv heads, blocks of the longest): rows beyond what one pass
# of a row's threads reads, 1024 of them where the rows fit the GPU at once, 256
# where there are more; rows of odd lengths, and shorter ones beside them
ROWS = [(2, 8, 2, 6001), (3, 4, 1, 4097), (1, 2, 1, 20000), (40, 16, 8, 2100), (77, 4, 4, 1025),
        (320, 1, 1, 4500)]


def _rows(b, h, hkv, n, d=64, bs=16):
    """Every sequence reads the same blocks in another order."""
    g = R.gen(b + n, "cuda")
    order = torch.stack([torch.randperm(n, generator=g, device="cuda") for _ in range(b)])
    blocks = [n - (i * 7) % 40 for i in range(b)]
    bounds = torch.randint(0, 100, (n, hkv, 2, d), generator=g, device="cuda")
    bounds = bounds.sort(2, descending=True).values.to(torch.int8)
    q = torch.randn(b, h, d, generator=g, device="cuda").half()
    sl = R.ints([k * bs - i % bs for i, k in enumerate(blocks)])
    return q, bounds, torch.ones(n, hkv, device="cuda"), order.int(), sl, blocks


@pytest.mark.parametrize("b,h,hkv,n", ROWS)
@pytest.mark.parametrize("sink,recent", [(40, 24), (0, 64), (64, 0), (1, 0)])
def test_nothing_left_to_choose(pa, b, h, hkv, n, sink, recent):
    """sinks + recents == max_selected: the scores do not matter."""
    q, bounds, bsc, tables, sl, blocks = _rows(b, h, hkv, n)
    want = torch.tensor([list(range(sink)) + list(range(k - recent, k)) for k in blocks],
                        dtype=torch.int32, device="cuda")[:, None].expand(-1, hkv, -1)
    for _ in range(10):
        lists, counts = _select(pa, q, bounds, bsc, tables, sl, 16, sink + recent, sink, recent)
        assert torch.equal(lists, want) and (counts == sink + recent).all()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("b,h,hkv,n", ROWS)
@pytest.mark.parametrize("kind", ["zero queries", "infinite scales", "bounds of zeros"])
def test_all_scores_equal(pa, b, h, hkv, n, kind):
    """The kept blocks, then the lowest positions."""
    q, bounds, bsc, tables, sl, blocks = _rows(b, h, hkv, n)
    if kind == "zero queries":
        q.zero_()
    elif kind == "infinite scales":
        bsc.fill_(math.inf)
    else:
        bounds.zero_()
    most, sink, recent = 50, 3, 5
    want = torch.tensor([list(range(most - recent)) + list(range(k - recent, k)) for k in blocks],
                        dtype=torch.int32, device="cuda")[:, None].expand(-1, hkv, -1)
    for _ in range(10):
        lists, counts = _select(pa, q, bounds, bsc, tables, sl, 16, most, sink, recent)
        assert torch.equal(lists, want) and (counts == most).all()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("b,h,hkv,n", ROWS[:1] + [(3, 8, 4, 300), (2, 4, 2, 1500)])
def test_scales_that_are_not_finite(pa, b, h, hkv, n):
    """Blocks whose bounds were never written may hold any bits: a scale of NaN
    of either sign or of an infinity counts as +inf, before every score, and
    never as a block that is kept anyway."""
    q, bounds, bsc, tables, sl, blocks = _rows(b, h, hkv, n)
    g = R.gen(3, "cuda")
    odd = torch.rand(n, hkv, generator=g, device="cuda")
    seen = torch.where(odd < 0.4, math.inf, bsc)           # what the definition sees
    bits = torch.full((n, hkv), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    bits[odd < 0.3] = 0x7F800001                           # NaN of other bits
    bits[odd < 0.2] = -1                                   # 0xFFFFFFFF, a negative NaN
    bits[odd < 0.1] = -0x800000                            # 0xFF800000, -inf
    spoiled = torch.where(odd < 0.4, bits.view(torch.float32), bsc)
    for most in (20, n // 2):                              # fewer and more than there are of them
        got = _select(pa, q, bounds, spoiled, tables, sl, 16, most, 2, 3)
        want = R.ref_select(q, bounds, seen, tables, sl, 16, most, 2, 3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    spoiled.view(torch.int32).fill_(-1)                    # every block
    got = _select(pa, q, bounds, spoiled, tables, sl, 16, 20, 2, 3)
    want = torch.tensor([list(range(17)) + list(range(k - 3, k)) for k in blocks],
                        dtype=torch.int32, device="cuda")
    assert torch.equal(got[0], want[:, None].expand(-1, hkv, -1))
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("e", [60, -60])
def test_scores_at_the_ends_of_the_scales(pa, e, sign):
    """Queries and blocks of the largest scale (scores of up to 2^140) and of the
    smallest (down to 2^-120): more blocks than are chosen, all scores distinct,
    positive or negative, and one block of infinite scale before them."""
    h, hkv, d, bs, n, most = 4, 2, 64, 16, 400, 150
    g = R.gen(5, "cuda")
    tables = torch.randperm(n, generator=g, device="cuda").int()[None].contiguous()
    steps = torch.arange(n, device="cuda") + 1
    bounds = torch.zeros(n, hkv, 2, d, dtype=torch.int8, device="cuda")
    for i in range(4):  # the sums are 127 * (1 .. n), in turn for each head
        part = (steps - 100 * i).clamp(0, 100)
        bounds[:, 0, :, i] = part[:, None].to(torch.int8)
        bounds[:, 1, :, d - 1 - i] = part.flip(0)[:, None].to(torch.int8)
    bsc = torch.full((n, hkv), 2.0 ** e, device="cuda")
    bsc[7, 0] = math.inf
    q = torch.full((1, h, d), sign * 127 * 2.0 ** e, device="cuda").to(torch.bfloat16)
    if e > 0:
        q[0, 1, 20], q[0, 2, 20] = math.inf, -math.inf         # met by codes of zero
    sl = R.ints([n * bs])
    got = _select(pa, q, bounds, bsc, tables, sl, bs, most, 0, 0)
    want = R.ref_select(q, bounds, bsc, tables, sl, bs, most, 0, 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int((tables[0] == 7).nonzero()) in got[0][0, 0].tolist()
