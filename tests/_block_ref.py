"""Plain 64-bit restatements of the block-scaled and block-sparse operators
(include/pa.h: pa_*_fp8_block, pa_update_block_bounds, pa_select_blocks,
pa_decode_sparse), request by request, and the inputs and tolerances of their
tests.  Nothing here shares code with the library."""
from __future__ import annotations

import math

import torch

E4M3_MAX, INT8_MAX = 448.0, 127.0


def scale_for(amax: torch.Tensor, top: float) -> torch.Tensor:
    """Smallest 2^e, e in [-60, 60], with amax <= top 2^e (61 if there were one
    is held to 60): found by trying every e."""
    out = torch.full_like(amax, 2.0 ** 60, dtype=torch.float64)
    for e in range(59, -61, -1):
        out[amax <= top * 2.0 ** e] = 2.0 ** e
    return out


def e4m3_table(device="cpu") -> torch.Tensor:
    """Value of each of the 256 codes (NaN at 0x7F and 0xFF)."""
    v = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        m = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(math.nan if c & 127 == 127 else -m if c & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device=device)


def e4m3_encode(x: torch.Tensor) -> torch.Tensor:
    """Nearest code, ties to the even one, magnitudes above 448 to 448."""
    x = x.double()
    mags = e4m3_table(x.device)[:127]
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a.nan_to_num(0.0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = mags[hi] - a, a - mags[lo]
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    pick = torch.where(torch.isnan(x), 127, pick)
    return (pick | torch.where(torch.signbit(x), 128, 0)).to(torch.uint8)


def requests(seq_lens, query_start_loc):
    qsl = query_start_loc.tolist()
    for r, length in enumerate(seq_lens.tolist()):
        yield r, length, qsl[r + 1] - qsl[r], qsl[r]


def ref_write(key, value, pool, scales, tables, seq_lens, query_start_loc, bs):
    """(codes, scales) after pa_reshape_and_cache_fp8_block."""
    pool, scales = pool.clone(), scales.clone()
    table = e4m3_table(pool.device)
    for r, length, q, row in requests(seq_lens, query_start_loc):
        start = length - q
        for j in range(start // bs, -(-length // bs) if q else 0):
            lo, hi = max(start, j * bs), min(length, j * bs + bs)
            blk, o, n = int(tables[r, j]), lo - j * bs, hi - lo
            for plane, src in enumerate((key, value)):
                x = src[row + lo - start:row + hi - start].double()
                a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((0, 2))
                s = scale_for(a, E4M3_MAX)
                if o:
                    was = scales[plane, blk].double()
                    s = torch.maximum(s, was)
                    held = pool[plane, blk, :o]
                    moved = e4m3_encode(table[held.long()] * (was / s)[None, :, None])
                    pool[plane, blk, :o] = torch.where((s > was)[None, :, None], moved, held)
                pool[plane, blk, o:o + n] = e4m3_encode(x / s[None, :, None])
                scales[plane, blk] = s.float()
    return pool, scales


def keys_of(pool, scales):
    """Key plane in 64 bits [NB, bs, Hkv, D]."""
    if scales is None:
        return pool[0].double()
    return e4m3_table(pool.device)[pool[0].long()] * scales[0].double()[:, None, :, None]


def ref_bounds(bounds, bounds_scale, pool, scales, tables, seq_lens, query_start_loc, bs):
    bounds, bounds_scale, keys = bounds.clone(), bounds_scale.clone(), keys_of(pool, scales)
    for r, length, q, _ in requests(seq_lens, query_start_loc):
        for j in range((length - q) // bs, -(-length // bs) if q else 0):
            blk = int(tables[r, j])
            k = keys[blk, :min(bs, length - j * bs)]
            fine = torch.isfinite(k).all(2).all(0)
            k = torch.where(fine[None, :, None], k, 0.0)
            s = scale_for(k.abs().amax((0, 2)), INT8_MAX)
            up = torch.ceil(k.amax(0) / s[:, None]).clamp(-INT8_MAX, INT8_MAX)
            low = torch.floor(k.amin(0) / s[:, None]).clamp(-INT8_MAX, INT8_MAX)
            bounds[blk, :, 0] = torch.where(fine[:, None], up, 0.0).to(torch.int8)
            bounds[blk, :, 1] = torch.where(fine[:, None], low, 0.0).to(torch.int8)
            bounds_scale[blk] = torch.where(fine, s, math.inf).float()
    return bounds, bounds_scale


def ref_select(q, bounds, bounds_scale, tables, seq_lens, bs, most, sink, recent):
    """A positive code meets the upper bound, a negative one the lower."""
    b, h, d = q.shape
    hkv = bounds.shape[1]
    x = q.double().view(b, hkv, h // hkv, d)
    a = torch.where(torch.isnan(x), 0.0, x.abs()).amax(-1)
    qs = scale_for(a, INT8_MAX)
    c = torch.round(torch.where(torch.isnan(x), 0.0, x) / qs[..., None]).clamp(-127, 127).long()
    lists = torch.full((b, hkv, most), -1, dtype=torch.int32, device=q.device)
    counts = torch.zeros(b, dtype=torch.int32, device=q.device)
    for s, length in enumerate(seq_lens.tolist()):
        n = -(-length // bs)
        counts[s] = min(n, most)
        for k in range(hkv):
            ids = tables[s, :n].long()
            up, low = bounds[ids, k, 0].long(), bounds[ids, k, 1].long()   # [n, D]
            cc = c[s, k][:, None]
            dots = torch.where(cc > 0, cc * up[None], cc * low[None]).sum(-1)
            score = (dots.double() * qs[s, k][:, None]).amax(0) if n else bounds_scale.new_zeros(0)
            bsc = bounds_scale[ids, k].double()
            score = torch.where(torch.isinf(bsc), math.inf, score * bsc.nan_to_num(posinf=0.0))
            # (kept first, then the score, then the position)
            score = score.tolist()
            order = sorted(range(n), key=lambda j: (not (j < sink or j >= n - recent),
                                                    -score[j], j))
            chosen = sorted(order[:most])
            lists[s, k, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return lists, counts


def ref_decode(q, pool, scales, tables, seq_lens, bs, scale, lists=None, list_lens=None):
    """(out, lse, weight) in 64 bits; `weight` [B, H, D] is sum_t p_t |v_t|, by
    which the tolerance goes, `reach` [B, H] the largest scale sum_d |q_d k_d|."""
    b, h, d = q.shape
    hkv = pool.shape[3]
    g = h // hkv
    out = torch.zeros(b, h, d, dtype=torch.float64, device=q.device)
    weight, reach = torch.zeros_like(out), torch.zeros(b, h, dtype=torch.float64, device=q.device)
    lse = torch.full((b, h), -math.inf, dtype=torch.float64, device=q.device)
    table = None if scales is None else e4m3_table(q.device)
    for s, length in enumerate(seq_lens.tolist()):
        for k in range(hkv):
            js = torch.arange(-(-length // bs), device=q.device)
            if lists is not None:
                js = lists[s, k, :int(list_lens[s])].long()
                js = js[(js >= 0) & (js < -(-length // bs))]
            ids = tables[s, js].long()
            ok = (ids >= 0) & (ids < pool.shape[1])
            kv = pool[:, ids.clamp(0, pool.shape[1] - 1), :, k]            # [2, n, bs, D]
            if scales is not None:
                kv = table[kv.long()] * scales[:, ids.clamp(0, pool.shape[1] - 1), k].double()[
                    ..., None, None]
            kv = torch.where(ok[None, :, None, None], kv.double(), 0.0)
            live = (js[:, None] * bs + torch.arange(bs, device=q.device) < length).flatten()
            kk, vv = kv.flatten(1, 2)[:, live]
            if not len(kk):
                continue
            qq = q[s, k * g:(k + 1) * g].double()
            a = qq @ kk.T * scale
            p = torch.softmax(a, -1)
            rows = slice(k * g, (k + 1) * g)
            out[s, rows], weight[s, rows] = p @ vv, p @ vv.abs()
            lse[s, rows] = torch.logsumexp(a, -1)
            reach[s, rows] = (qq.abs() @ kk.abs().T * abs(scale)).amax(-1)
    return out, lse, weight, reach


def check_decode(got, ref, half_products: bool, two_parts: bool, lse=None):
    """The kernel's error is at most
      eps(out) |ref|        rounding of the output, eps = half a step relative
                            (2^-11 fp16, 2^-8 bf16), plus fp16's subnormal step
      + eps_p W             rounding of the probabilities: one part 2^-11 in
                            halves; two parts 2^-22 in halves, 2^-16 in bf16
      + 2 d W               each probability is off by a factor within 1 +- d,
                            and so is the normaliser
    with W = sum p |v| and d = 2^-21 (1 + 2 R): exp2 of an fp32 argument, whose
    rounding and products' sums over at most 128 channels (chains of 8 steps,
    each within 2^-23 of the sum of magnitudes so far) are within 2^-20 R for
    scores whose products' magnitudes sum to R."""
    out, ref_lse, weight, reach = ref
    dtype = got.dtype
    eps = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    eps_p = (2.0 ** -22 if half_products else 2.0 ** -16) if two_parts else 2.0 ** -11
    d = 2.0 ** -21 * (1 + 2 * reach[..., None])
    err = (got.double() - out).abs()
    bound = (eps * (out.abs() + (eps_p + 2 * d) * weight) + (eps_p + 2 * d) * weight +
             2.0 ** -25)
    assert torch.isfinite(got.double()).all()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3g} times the bound"
    if lse is not None:
        empty = torch.isinf(ref_lse)
        assert torch.equal(empty, torch.isinf(lse)) and (lse[empty] < 0).all()
        # log of a sum within 1 +- d, plus the fp32 rounding of the result
        lb = d[..., 0] * 2 + 2.0 ** -22 * (1 + ref_lse.abs())
        e = (lse.double() - ref_lse).abs()[~empty]
        assert (e <= lb[~empty]).all(), (e / lb[~empty]).max()
    return worst


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def make_tables(lens, bs, extra=3, device="cuda", seed=0, width=0):
    """Block tables dealt from a random order of the pool's blocks, -1 behind a
    sequence's last; (tables, number of blocks)."""
    n = [-(-v // bs) for v in lens]
    nb = sum(n) + extra
    order = torch.randperm(nb, generator=gen(seed, "cpu")).tolist()
    t = torch.full((len(lens), max([1, width] + n)), -1, dtype=torch.int32)
    at = 0
    for s, k in enumerate(n):
        t[s, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
    return t.to(device), nb


def starts(q_lens, device="cuda"):
    return torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32,
                        device=device)


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def make_pool(nb, bs, hkv, d, dtype, eight, device="cuda", seed=0, spread=0.0):
    """A pool of normal values; spread > 0 gives every (plane, block, head) its
    own magnitude 2^(spread * normal).  (pool, kv_scales or None)."""
    g = gen(seed, device)
    x = torch.randn(2, nb, bs, hkv, d, generator=g, device=device)
    if spread:
        x *= torch.exp2(spread * torch.randn(2, nb, 1, hkv, 1, generator=g, device=device))
    x = x.to(dtype)
    if not eight:
        return x, None
    s = scale_for(x.double().abs().amax((2, 4)), E4M3_MAX)
    return e4m3_encode(x.double() / s[:, :, None, :, None]), s.float()


def poison_tails(pool, tables, lens, bs):
    """NaN in every row that no sequence owns: the rest of last blocks and the
    free blocks."""
    own = torch.zeros(pool.shape[1], bs, dtype=torch.bool)
    for s, length in enumerate(lens):
        for j in range(-(-length // bs)):
            own[int(tables[s, j]), :min(bs, length - j * bs)] = True
    pool[:, ~own.to(pool.device)] = 0x7F if pool.dtype == torch.uint8 else math.nan
