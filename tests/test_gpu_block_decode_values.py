"""Decode over an e4m3 pool and over listed blocks where the values of a row
cancel, so that what the probabilities are rounded to shows in the output."""
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
    return torch.full((pa.pa_block_decode_workspace_size(h, hkv, d),), 0xFF, dtype=torch.uint8,
                      device="cuda")


def _cancelling(lens, h, hkv, d, bs, dtype, eight, seed):
    """Tokens in pairs of opposite values whose keys differ in one channel, by
    which their scores differ by about 2^-8: the output is a small part of
    sum p |v|."""
    tables, nb = R.make_tables(lens, bs, seed=seed)
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, eight, seed=seed)
    g = R.gen(seed, "cuda")
    q = torch.randn(len(lens), h, d, generator=g, device="cuda")
    q[..., 0] = 2.0 ** -6 * (1 + torch.rand(len(lens), h, generator=g, device="cuda"))
    pool[0, :, 1::2, :, 1:] = pool[0, :, ::2, :, 1:]
    sign = 0x80 if eight else None
    pool[1, :, 1::2] = pool[1, :, ::2] ^ sign if eight else -pool[1, :, ::2]
    return q.to(dtype), pool, scales, tables, R.ints(lens)


@pytest.mark.parametrize("h,hkv,d,bs", [(8, 2, 128, 16), (16, 2, 64, 32), (4, 4, 128, 32)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("eight", [True, False])
def test_probabilities_keep_two_parts(pa, h, hkv, d, bs, dtype, eight):
    lens = [2, 4, 8, 14, 32, 6, 1000]
    q, pool, scales, tables, sl = _cancelling(lens, h, hkv, d, bs, dtype, eight, 3)
    ws, scale = _workspace(pa, h, hkv, d), 1 / math.sqrt(d)
    blocks = [-(-v // bs) for v in lens]
    lists = torch.full((len(lens), hkv, max(blocks)), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(blocks):
        lists[s, :, :n] = torch.arange(n, device="cuda")
    ref = R.ref_decode(q, pool, scales, tables, sl, bs, scale)
    outs = [torch.empty_like(q)]
    pa.pa_decode_sparse(outs[0], q, pool, tables, sl, lists, R.ints(blocks), scale, bs, ws,
                        kv_scales=scales)
    if eight:
        outs.append(torch.empty_like(q))
        pa.pa_decode_fp8_block(outs[1], q, pool, scales, tables, sl, scale, bs, max(lens), ws)
    for out in outs:
        R.check_decode(out, ref, half_products=eight or dtype == torch.float16, two_parts=True)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("eight", [True, False])
@pytest.mark.parametrize("length", [8176, 8192, 524288])
def test_long_runs_do_not_lose_weight(pa, length, eight, dtype):
    """Values of 1 in a run of tokens that one warp sums: the output is 1.

    Additions that round to nearest are off by at most 2^-24 of the sum so far,
    with either sign alike: over the 32768 of the longest run their sum has a
    standard deviation of at most 2^-24 sqrt(32768 / 3) = 6.3e-6, and the
    normaliser's the same.  An e4m3 pool's sums of up to 512 tiles are truncated,
    by at most 2^-23 of the sum so far in each of a tile's two products: at most
    2^-14 = 6.1e-5 of a sum that grows evenly.  The nearest 16-bit number is 1 as
    long as all that is within 2^-12 = 2.4e-4 (fp16), 2^-9 (bf16)."""
    b, h, hkv, d, bs, nb = 304, 8, 8, 128, 16, 64
    if length > 10 ** 5:
        b, bs = 152, 32
    g = R.gen(4, "cuda")
    pool, scales = R.make_pool(nb, bs, hkv, d, dtype, eight, seed=4)
    pool[1] = 0x38 if eight else 1.0
    if eight:
        scales[1] = 1.0
    # a few blocks in random order, so that no table of that length needs a pool
    n = length // bs
    tables = torch.randint(0, nb, (b, n), generator=g, device="cuda").int()
    sl = torch.full((b,), length, dtype=torch.int32, device="cuda")
    q = torch.randn(b, h, d, generator=g, device="cuda").to(dtype)
    out, ws = torch.zeros_like(q), _workspace(pa, h, hkv, d)
    if eight:
        pa.pa_decode_fp8_block(out, q, pool, scales, tables, sl, 0.05, bs, length, ws)
    else:
        lists = torch.arange(n, dtype=torch.int32, device="cuda").expand(b, hkv, n).contiguous()
        counts = torch.full((b,), n, dtype=torch.int32, device="cuda")
        pa.pa_decode_sparse(out, q, pool, tables, sl, lists, counts, 0.05, bs, ws)
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    assert (out == 1.0).all(), (out.double() - 1).abs().max()
