"""Plain 64-bit restatement of linear attention with a decay for each head
(include/pa.h: pa_linear_decode, pa_linear_prefill), token by token, and the inputs
and tolerances of its tests.  Nothing here shares code with the library."""
from __future__ import annotations

import math

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def ref_linear(q, k, v, log_decay, states, src, dst, starts, scale):
    """(out, states, magnitude of out, magnitude of states) in 64 bits.  The
    magnitudes are the same sums over absolute values; rows and states that the call
    does not write are None in `wrote` terms: out rows stay NaN, states stay."""
    t, h, d = q.shape
    hkv = k.shape[1]
    q, k, v, g = q.double(), k.double(), v.double(), log_decay.double()
    out = torch.full((t, h, d), math.nan, dtype=torch.float64, device=q.device)
    mag, new = out.clone(), states.double().clone()
    new_mag = new.abs()
    starts = starts.tolist()
    for s in range(len(starts) - 1):
        to, of = int(dst[s]), int(src[s])
        if to < 0:
            continue
        S = states[of].double().clone() if 0 <= of < len(states) else torch.zeros(
            hkv, d, d, dtype=torch.float64, device=q.device)
        M = S.abs()
        for i in range(starts[s], starts[s + 1]):
            a = torch.exp(g if g.dim() == 1 else g[i])[:, None, None]
            kv = k[i][:, :, None] * v[i][:, None, :]
            S, M = a * S + kv, a * M + kv.abs()
            qi = q[i].view(hkv, h // hkv, d) * scale
            out[i] = (qi @ S).view(h, d)
            mag[i] = (qi.abs() @ M).view(h, d)
        if to < len(states):
            new[to], new_mag[to] = S, M
    return out, new, mag, new_mag


# A value that enters a product as a rounded 16-bit part and the rounded remainder is
# off by (eps / 2)^2 of its size: 2^-16 with bf16, 2^-22 with fp16.  An output's sum
# has at most two such values behind a term (a state that was made of decayed values,
# then split itself).  In fp32: a decay's exponent is a sum of at most 7 levels, off by
# 7 * 2^-24 * |x|, and |x| e^-|x| <= 0.37 (within a block of 32 tokens it is a difference
# of two sums u from the block's first token, each off by 2^-24 |u| a level: with the
# decays of `inputs` |u| is at most 23 and 6 at the mean, and the levels' errors have both
# signs); exponentials 2^-22; a product's 8 steps of 16 terms that the matrix unit adds
# with truncation, 2^-23 each, twice: below 2^-18 in all.
SLACK = {torch.bfloat16: 2.0 ** -15 + 2.0 ** -18, torch.float16: 2.0 ** -21 + 2.0 ** -18}


def check_out(got, ref, mag, what=""):
    """|got - ref| within half a step of the output's type and the slack above."""
    live = ~torch.isnan(mag)
    half = torch.finfo(got.dtype).eps / 2
    least = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    slack = SLACK[got.dtype] * mag
    tol = half * (ref.abs() + slack) + slack + least
    err = (got.double() - ref).abs()
    bad = live & ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol)[live].max()),
                           bad.nonzero()[:4].tolist())


def check_states(got, ref, mag, dtype, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= SLACK[dtype] * mag + 2.0 ** -24 * ref.abs())
    assert not bad.any(), (what, int(bad.sum()), float((err / mag.clamp(min=1e-30)).max()),
                           bad.nonzero()[:4].tolist())
    # Roundings of both signs average: the root mean square of two 8-bit roundings in a
    # row, each uniform in half a step, is below 2^-16 / 3
    norm = float(ref.norm())
    assert norm == 0 or float((got.double() - ref).norm()) <= 2.0 ** -17 * norm, what


def inputs(lens, heads, kv_heads, d, dtype, decay="token", seed=0, fresh=(), device="cuda",
           spare=1, fused=False, tail=0):
    """Random inputs; sequence i starts from nothing if i is in `fresh`.  `fused`: q, k
    and v are slices of one projection's rows.  `tail`: token rows behind the last."""
    g = torch.Generator().manual_seed(seed)
    t, b, dt = sum(lens) + tail, len(lens), DTYPES[dtype]
    wide = (heads + 2 * kv_heads) * d
    x = torch.randn(t, wide, generator=g).to(dt).to(device)
    q, k, v = x.split([heads * d, kv_heads * d, kv_heads * d], dim=1)
    q, k, v = q.view(t, heads, d), k.view(t, kv_heads, d), v.view(t, kv_heads, d)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rate = -torch.exp2(-8.0 * (torch.arange(kv_heads) + 1) / kv_heads)
    if decay == "token":
        rate = rate * 2 * torch.rand(t, kv_heads, generator=g)
    n = 2 * b + spare
    deal = torch.randperm(n, generator=g).int()
    src, dst = deal[:b].clone(), deal[b:2 * b].clone()
    for i in (i for i in fresh if i < b):
        src[i] = -1
    starts = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32)
    return dict(q=q, k=k, v=v, log_decay=rate.float().to(device),
                states=(4 * torch.randn(n, kv_heads, d, d, generator=g)).to(device),
                src=src.to(device), dst=dst.to(device), starts=starts.to(device),
                scale=1.0 / math.sqrt(d))
