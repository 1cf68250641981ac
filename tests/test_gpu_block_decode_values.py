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
