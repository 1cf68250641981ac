"""The cache-side block operators on the GPU against their 64-bit restatement:
the write into an e4m3 pool with block scales and the key bounds, bit-exact."""
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


# (cached tokens after the call, new ones) of each request
SHAPES = {
    "steps": ([1, 16, 17, 31, 32, 33, 200], [1] * 7),
    "prompts": ([1, 15, 16, 47, 130], [1, 15, 16, 47, 130]),
    "chunks": ([40, 61, 300, 18, 16], [7, 45, 101, 2, 0]),
}


def _write(pa, name, dtype, d, hkv, bs, seed, spoil=None, strided=False, loud=0.0):
    lens, new = SHAPES[name]
    tables, nb = R.make_tables(lens, bs, seed=seed)
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, True, seed=seed, spread=1.0)
    qsl = R.starts(new)
    g = R.gen(seed + 1, "cuda")
    tokens = sum(new) + 2                       # two rows behind the last request
    kv = torch.randn(tokens, 2, hkv, d, generator=g, device="cuda")
    kv = (kv * torch.exp2(loud * torch.randn(tokens, 2, hkv, 1, generator=g, device="cuda")))
    kv = kv.to(dtype)
    if spoil is not None:
        spoil(kv)
    key, value = (kv[:, 0], kv[:, 1]) if strided else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
    want = R.ref_write(key, value, pool, scales, tables, R.ints(lens), qsl, bs)
    pa.pa_reshape_and_cache_fp8_block(key, value, pool, scales, tables, R.ints(lens), qsl, bs,
                                      max(new))
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    assert torch.equal(pool, want[0])
    assert torch.equal(scales, want[1])


@pytest.mark.parametrize("d,hkv,bs", [(128, 8, 16), (128, 3, 32), (64, 4, 16), (64, 1, 32)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("name", list(SHAPES))
def test_write_bit_exact(pa, name, dtype, d, hkv, bs):
    _write(pa, name, dtype, d, hkv, bs, seed=3, strided=hkv == 8, loud=2.0)


def test_write_non_finite_and_extreme_values(pa):
    def spoil(kv):
        kv[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 5.0])
        kv[1, 1, 1] = 0.0                          # a head of zeros
        kv[2, 0, 0] = math.nan                     # no finite value at all
        kv[3, 0, 1, 7] = -0.0
        kv[4, 1, 0, 3] = 3e38                      # above 448 * 2^60: saturates
        kv[5, 0, 0] = 1e-30                        # below 2^-60: code 0
    _write(pa, "prompts", torch.bfloat16, 128, 2, 16, seed=5, spoil=spoil)


def test_write_scales_at_the_borders(pa):
    """448 * 2^e itself takes 2^e; the next value up takes 2^(e+1)."""
    def spoil(kv):
        kv *= 0.01
        for i, v in enumerate((448.0, 450.0, 447.0, 28.0, 28.125, 1.75, 1.7578125)):
            kv[i, 0, 0, 0] = v
    _write(pa, "steps", torch.bfloat16, 64, 2, 16, seed=6, spoil=spoil)


def test_write_grows_a_scale_step_by_step(pa):
    """Tokens of rising magnitude appended one at a time: the block's earlier
    rows follow its scale, and a second call with the same token changes
    nothing."""
    d, hkv, bs = 128, 2, 16
    tables, nb = R.make_tables([bs], bs)
    pool, scales = R.make_pool(nb, bs, hkv, d, torch.float16, True)
    for t in range(bs):
        x = (torch.randn(1, hkv, d, generator=R.gen(t, "cuda"), device="cuda") * 2.0 ** (t % 7))
        x = x.half()
        args = (x, -x, pool, scales, tables, R.ints([t + 1]), R.starts([1]), bs)
        want = R.ref_write(*args)
        for _ in range(2):
            pa.pa_reshape_and_cache_fp8_block(*args, 1)
            assert torch.equal(pool, want[0]) and torch.equal(scales, want[1])


def test_write_skips_and_flags_bad_requests(pa):
    bs, hkv, d = 16, 2, 64
    lens = [20, 20, 20, 20]
    tables, nb = R.make_tables(lens, bs)
    tables[1, 1] = nb                              # outside the pool
    pool, scales = R.make_pool(nb, bs, hkv, d, torch.float16, True)
    kv = torch.randn(8, hkv, d, device="cuda", dtype=torch.float16)
    qsl = R.starts([2, 2, 2, 2])
    seen = R.ints([20, 20, 1, 4000])               # shorter than its new tokens; past its table
    good, good_s = R.ref_write(kv, kv, pool, scales, tables, R.ints([20, 0, 0, 0]),
                               R.starts([2, 0, 0, 0]), bs)
    pa.pa_reshape_and_cache_fp8_block(kv, kv, pool, scales, tables, seen, qsl, bs, 2)
    flags = pa.pa_device_errors(clear=True)
    assert flags & pa.DEVERR_BLOCK_ID and flags & pa.DEVERR_SEQ_LEN
    assert torch.equal(pool, good) and torch.equal(scales, good_s)
    # more new tokens than max_query_len: every request is skipped
    pa.pa_reshape_and_cache_fp8_block(kv, kv, pool, scales, tables, R.ints(lens), qsl, bs, 1)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    assert torch.equal(pool, good)


def test_write_takes_a_slice_of_a_wider_table(pa):
    bs, hkv, d = 16, 4, 128
    lens, new = [33, 5], [9, 5]
    wide, nb = R.make_tables(lens, bs, width=11)
    tables = wide[:, :3]
    pool, scales = R.make_pool(nb, bs, hkv, d, torch.bfloat16, True)
    x = torch.randn(14, hkv, d, device="cuda", dtype=torch.bfloat16)
    want = R.ref_write(x, x, pool, scales, tables, R.ints(lens), R.starts(new), bs)
    pa.pa_reshape_and_cache_fp8_block(x, x, pool, scales, tables, R.ints(lens), R.starts(new), bs,
                                      100)
    assert torch.equal(pool, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("d,hkv,bs", [(128, 8, 16), (128, 3, 32), (64, 4, 32), (64, 9, 16)])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_bounds_bit_exact(pa, name, kind, d, hkv, bs):
    lens, new = SHAPES[name]
    dtype = torch.bfloat16 if kind == "bf16" else torch.float16
    tables, nb = R.make_tables(lens, bs, seed=9)
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, kind == "e4m3", seed=9, spread=2.0)
    R.poison_tails(pool, tables, lens, bs)
    g = R.gen(1, "cuda")
    bounds = torch.randint(-128, 128, (nb, hkv, 2, d), generator=g, device="cuda").to(torch.int8)
    bsc = torch.rand(nb, hkv, generator=g, device="cuda")
    want = R.ref_bounds(bounds, bsc, pool, scales, tables, R.ints(lens), R.starts(new), bs)
    pa.pa_update_block_bounds(bounds, bsc, pool, tables, R.ints(lens), R.starts(new), bs, max(new),
                              kv_scales=scales)
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    assert torch.equal(bounds, want[0])
    assert torch.equal(bsc, want[1])


@pytest.mark.parametrize("kind", ["fp16", "bf16", "e4m3"])
def test_bounds_of_odd_keys(pa, kind):
    """Not finite, zero, one huge and tiny ones; 127 * 2^e and the next value."""
    bs, hkv, d = 16, 2, 128
    lens = [48, 16]
    dtype = torch.bfloat16 if kind == "bf16" else torch.float16
    tables, nb = R.make_tables(lens, bs)
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, kind == "e4m3")
    b = tables[0].tolist()
    if kind == "e4m3":
        pool[0, b[0], 3, 1, 5] = 0x7F
        pool[0, b[1], :, 0] = 0
    else:
        pool[0, b[0], 3, 1, 5] = math.nan
        pool[0, b[0], 15, 0, 127] = -math.inf
        pool[0, b[1], :, 0] = 0
        pool[0, b[1], 0, 1, 0] = 127.0 * 4
        pool[0, b[2], 0, 1, 0] = 127.5 * 4 if kind == "fp16" else 128.0 * 4
        pool[0, b[2], 0, 0, 0] = 6e4 if kind == "fp16" else 3e38
        pool[0, tables[1, 0]] = 0.0
        pool[0, tables[1, 0], 2, 0, 9] = -6e-8 if kind == "fp16" else -1e-35
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.zeros(nb, hkv, device="cuda")
    want = R.ref_bounds(bounds, bsc, pool, scales, tables, R.ints(lens), R.starts(lens), bs)
    pa.pa_update_block_bounds(bounds, bsc, pool, tables, R.ints(lens), R.starts(lens), bs, 48,
                              kv_scales=scales)
    assert torch.equal(bounds, want[0]) and torch.equal(bsc, want[1])


def test_bounds_bound_every_key(pa):
    """upper * scale and lower * scale enclose the keys of the pool."""
    bs, hkv, d, lens = 16, 8, 128, [16 * 20]
    tables, nb = R.make_tables(lens, bs)
    pool, _ = R.make_pool(nb, bs, hkv, d, torch.bfloat16, False)
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.zeros(nb, hkv, device="cuda")
    pa.pa_update_block_bounds(bounds, bsc, pool, tables, R.ints(lens), R.starts(lens), bs, 320)
    ids = tables[0].long()
    k, s = pool[0, ids].double(), bsc[ids].double()[:, None, :, None]
    assert (k <= bounds[ids, :, 0].double()[:, None] * s).all()
    assert (k >= bounds[ids, :, 1].double()[:, None] * s).all()
