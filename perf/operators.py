"""The operators of a long-context decode step that reads fewer bytes: their
calls, their plain forms and the sizes at which they are measured.

Five operators over the paged pool [2, num_blocks, block_size, num_kv_heads,
head_size] (plane 0 keys, plane 1 values):

  write8   append new tokens to a pool held in e4m3 with one scale for each
           (plane, block, kv head)
  decode8  decode attention over such a pool
  bounds   per (block, kv head) and channel, the largest and smallest key, in
           8 bits with one scale for each (block, kv head)
  select   the blocks of every (sequence, kv head) whose keys can score
           highest for the step's queries, by those bounds
  sparse   decode attention over the selected blocks, of a 16-bit pool or of
           a pool as write8 keeps it

Every scale is a power of two: pow2_scale(amax, top) is the smallest 2^e with
amax <= top * 2^e, e held to [-60, 60].  Codes times such a scale are exact, so
a block whose scale grows keeps the values it holds (but for e4m3's subnormal
end), and the scores of `select` are whole numbers times powers of two, exact in
32 bits whatever the order of the sum: the chosen blocks have one right answer.
"""
import math
import random

import torch

own = False

_DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
_TOP8 = 448.0      # largest e4m3 magnitude
_TOPB = 127.0      # largest magnitude of the bounds' and the queries' codes


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(name, op, seqs, lens, lo, hi, heads, kv_heads, head_size, block_size, dtype, **more):
    c = dict(op=op, seqs=seqs, lens=lens, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads,
             head_size=head_size, block_size=block_size, dtype=dtype, lens_seed=1)
    if name:
        c["name"] = name
    c.update(more)
    return c


def listed():
    return [
        # one decode step's cache write of 256 running requests (grouped queries)
        _case("write8 step 256", "write8", 256, "lognormal", 16, 4096, 32, 8, 128, 16, "bf16",
              new_lo=1, new_hi=1),
        # the cache write of 16 prompts, half of them continued chunks
        _case("write8 prompts", "write8", 16, "uniform", 2048, 4096, 32, 32, 128, 16, "fp16",
              new_lo=256, new_hi=2048),
        # the smallest decode: four short requests of a small model
        _case("decode8 tiny", "decode8", 4, "ladder", 1, 64, 4, 4, 64, 16, "fp16"),
        # decode of 64 requests, one kv head for each query head
        _case("decode8 mha 64", "decode8", 64, "uniform", 128, 2048, 32, 32, 128, 16, "fp16"),
        # decode of 256 requests of very different lengths, grouped queries
        _case("decode8 gqa 256", "decode8", 256, "lognormal", 16, 4096, 32, 8, 128, 16, "bf16"),
        # decode over 8 contexts of 131072 tokens
        _case("decode8 long", "decode8", 8, "equal", 131072, 131072, 64, 8, 128, 32, "bf16"),
        # the step's refresh of the last block's bounds, 16-bit pool
        _case("bounds step 256", "bounds", 256, "lognormal", 16, 4096, 32, 8, 128, 16, "bf16",
              new_lo=1, new_hi=1, pool="16bit"),
        # the bounds of 16 prompts in the 8-bit pool
        _case("bounds prompts", "bounds", 16, "uniform", 2048, 4096, 32, 32, 128, 16, "fp16",
              new_lo=256, new_hi=2048, pool="8bit"),
        # a few requests of medium length: 64 of at most 512 blocks
        _case("select small", "select", 4, "uniform", 2048, 8192, 32, 8, 128, 16, "fp16",
              select=64, sink=1, recent=2),
        # 8 contexts of 131072 tokens: 128 of 4096 blocks
        _case("select long", "select", 8, "equal", 131072, 131072, 64, 8, 128, 32, "bf16",
              select=128, sink=1, recent=2),
        # attention over those 128 blocks of a 16-bit pool
        _case("sparse long 16bit", "sparse", 8, "equal", 131072, 131072, 64, 8, 128, 32, "bf16",
              select=128, pool="16bit"),
        # 64 requests of ragged length over 64 blocks each of an 8-bit pool
        _case("sparse ragged 8bit", "sparse", 64, "uniform", 500, 16384, 32, 8, 128, 16, "fp16",
              select=64, pool="8bit"),
    ]


_HEADS = [(4, 4), (8, 1), (16, 8), (12, 3), (32, 32), (32, 8), (64, 8), (32, 16), (6, 6), (40, 5)]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write8", "decode8", "bounds", "select", "sparse"])
    heads, kv_heads = rng.choice(_HEADS)
    d, bs = rng.choice([64, 128, 128]), rng.choice([16, 16, 32])
    more = {}
    hi = _spread(rng, {"select": 2048, "sparse": 64}.get(op, 8), 131072)
    if op in ("write8", "bounds"):
        hi = _spread(rng, 4, 8192)
        more["new_lo"] = 1
        more["new_hi"] = rng.choice([1, min(hi, _spread(rng, 1, 2048))])
    # at most the tokens and rows of the largest listed cases
    room = (64 << 20 if op in ("write8", "bounds") else 1 << 30) // (hi * kv_heads * d)
    seqs = max(1, min(_spread(rng, 1, 256), room))
    if op in ("bounds", "sparse"):
        more["pool"] = rng.choice(["16bit", "8bit"])
    if op in ("select", "sparse"):
        more["select"] = _spread(rng, 4, 256)
    if op == "select":  # fewer than there are, or there is nothing to choose
        more["select"] = max(4, min(more["select"], hi // bs // 16))
    if op == "select":
        more.update(sink=rng.choice([0, 1, 2]), recent=rng.choice([0, 1, 2]))
    kind = rng.choice(["uniform", "equal"] if op == "select" else
                      ["uniform", "lognormal", "equal"])
    lo = max(more.get("new_hi", 1), hi if kind == "equal" else max(1, hi // 8))
    if op == "select" and kind == "uniform" and seqs >= 8:
        lo = 1  # some requests shorter than the selection
    c = _case("", op, seqs, kind, min(lo, hi), hi, heads, kv_heads, d, bs,
              rng.choice(["fp16", "bf16"]), **more)
    c["lens_seed"] = rng.randrange(1 << 20)
    return c


def _lens(case):
    """(tokens in the cache, of them new) of every sequence, by the case alone."""
    r = random.Random(case["lens_seed"])
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if case["lens"] == "ladder":
        lens = [max(lo, hi * i // max(1, n - 1) + (1 if 0 < i < n - 1 else 0)) for i in range(n)]
        lens = [min(hi, v) for v in lens]
    elif case["lens"] == "lognormal":
        mid = math.log(max(1.0, hi / 8))
        lens = [min(hi, max(lo, int(round(math.exp(r.gauss(mid, 1.0)))))) for _ in range(n)]
    else:
        lens = [r.randint(lo, hi) for _ in range(n)]
    a, b = case.get("new_lo", 1), case.get("new_hi", 1)
    new = [min(v, r.randint(a, b)) for v in lens]
    if b > 1:  # every other prompt is a whole one, the rest continue
        lens = [q if i % 2 == 0 else v for i, (v, q) in enumerate(zip(lens, new))]
    return lens, new


def _blocks(case, lens):
    return [-(-v // case["block_size"]) for v in lens]


def _touched(case, lens, new):
    bs = case["block_size"]
    return sum((v - 1) // bs - (v - q) // bs + 1 for v, q in zip(lens, new) if q)


def work(case):
    lens, new = _lens(case)
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_size"], case["block_size"]
    row, b, nb = hkv * d, case["seqs"], sum(_blocks(case, lens))
    qo = 2 * b * h * d * 2
    if case["op"] == "write8":
        t = sum(new)
        # new rows read in 16 bits and written in 8, the touched blocks' scales
        return {"bytes": 2 * t * row * 3 + 2 * 8 * _touched(case, lens, new) * hkv + 8 * b,
                "flops": 4 * t * row}
    if case["op"] == "bounds":
        bs_rows = sum(v - (v - q) // bs * bs for v, q in zip(lens, new) if q)
        n = _touched(case, lens, new)
        wide = 2 if case["pool"] == "16bit" else 1
        return {"bytes": bs_rows * row * wide + n * hkv * (2 * d + 4) + 8 * b,
                "flops": 3 * bs_rows * row}
    if case["op"] == "decode8":
        return {"bytes": 2 * sum(lens) * row + 8 * nb * hkv + 4 * nb + 4 * b + qo,
                "flops": 4 * sum(lens) * h * d}
    if case["op"] == "select":
        k = sum(min(n, case["select"]) for n in _blocks(case, lens))
        return {"bytes": nb * hkv * (2 * d + 4) + 4 * nb + qo // 2 + 4 * k * hkv + 8 * b,
                "flops": 2 * nb * h * 2 * d}
    k = [min(n, case["select"]) for n in _blocks(case, lens)]
    tokens = sum(min(n * bs, v) for n, v in zip(k, lens))
    wide = 2 if case["pool"] == "16bit" else 1
    return {"bytes": 2 * tokens * row * wide + (8 * sum(k) * hkv if wide == 1 else 0) +
            8 * sum(k) * hkv + 4 * b + qo, "flops": 4 * tokens * h * d}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _pow2_scale(amax, top):
    """Smallest 2^e with amax <= top * 2^e, e in [-60, 60] (float32; amax >= 0)."""
    m, e = torch.frexp(amax)
    tm, te = math.frexp(top)
    e = (e - te + (m > tm).to(torch.int32)).clamp(-60, 60)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).to(torch.int32)
    return ((e + 127) << 23).view(torch.float32)


def _finite_amax(x, dims):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dims)


def _e4m3(x):
    return x.clamp(-_TOP8, _TOP8).to(torch.float8_e4m3fn).view(torch.uint8)


def _value8(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _span(s):
    """Blocks of every request that its new tokens reach: their physical ids
    [R, N], the tokens' positions [R, N, bs], and which of them are new, old or
    past the end; N covers the longest request."""
    bs, length, new = s["block_size"], s["seq_lens"].long(), s["new_lens"]
    start = length - new
    n = (s["max_query_len"] + bs - 2) // bs + 1
    dev = length.device
    j = (start // bs)[:, None] + torch.arange(n, device=dev)
    p = j[..., None] * bs + torch.arange(bs, device=dev)
    touched = (j * bs < length[:, None]) & (new > 0)[:, None]
    phys = s["block_tables"].long().gather(1, j.clamp(max=s["block_tables"].shape[1] - 1))
    phys = torch.where(touched, phys, 0)
    first = start[:, None, None]
    here = touched[..., None]
    return phys, p, here & (p >= first) & (p < length[:, None, None]), here & (p < first), touched


def _plain_write8(s):
    pool, scales = s["kv_cache"], s["kv_scales"]
    phys, p, new, old, touched = _span(s)
    start = s["seq_lens"].long() - s["new_lens"]
    row = (s["query_start_loc"].long()[:-1, None, None] + p - start[:, None, None])
    row = row.clamp(0, s["key"].shape[0] - 1)
    x = torch.stack((s["key"], s["value"]))[:, row].float()          # [2, R, N, bs, Hkv, D]
    x = torch.where(new[None, ..., None, None], x, 0.0)
    scale = _pow2_scale(_finite_amax(x, (3, 5)), _TOP8)               # [2, R, N, Hkv]
    before = scales[:, phys]
    scale = torch.where(old.any(2)[None, ..., None], torch.maximum(scale, before), scale)
    wide = scale[:, :, :, None, :, None]
    held = _e4m3(_value8(pool[:, phys]) * (before / scale)[:, :, :, None, :, None])
    codes = torch.where(new[None, ..., None, None], _e4m3(x / wide), held)
    r, n, o = (new | old).nonzero(as_tuple=True)
    pool[:, phys[r, n], o] = codes[:, r, n, o]
    r, n = touched.nonzero(as_tuple=True)
    scales[:, phys[r, n]] = scale[:, r, n]
    return pool.view(torch.float8_e4m3fn), scales


def _attend(q, k, v, live, scale):
    """q [B, Hkv, G, D], k and v [B, Hkv, L, D], live [B, Hkv, L]; fp32."""
    live = live[:, :, None, :]
    s = torch.where(live, q @ k.transpose(2, 3) * scale, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(live, torch.exp(s - m), 0.0)
    o = p @ torch.where(live.transpose(2, 3), v, 0.0)
    z = p.sum(-1, keepdim=True)
    return torch.where(live.any(-1, keepdim=True), o / z, 0.0)


def _grouped(q, kv_heads):
    return q.float().view(q.shape[0], kv_heads, -1, q.shape[2])


def _plain_decode8(s):
    pool, scales, q = s["kv_cache"], s["kv_scales"], s["q"]
    hkv, d = pool.shape[3], pool.shape[4]
    t = s["block_tables"].long().clamp(min=0)
    k = _value8(pool[0][t]) * scales[0][t][:, :, None, :, None]       # [B, MB, bs, Hkv, D]
    v = _value8(pool[1][t]) * scales[1][t][:, :, None, :, None]
    k, v = (x.flatten(1, 2).transpose(1, 2) for x in (k, v))
    live = torch.arange(k.shape[2], device=q.device) < s["seq_lens"][:, None]
    o = _attend(_grouped(q, hkv), k, v, live[:, None].expand(-1, hkv, -1), s["scale"])
    return o.view(-1, q.shape[1], d).to(q.dtype)


def _plain_bounds(s):
    pool, bs = s["kv_cache"], s["block_size"]
    phys, p, new, old, touched = _span(s)
    k = pool[0][phys]                                                 # [R, N, bs, Hkv, D]
    if s["kv_scales"] is not None:
        k = _value8(k) * s["kv_scales"][0][phys][:, :, None, :, None]
    k, live = k.float(), (new | old)[..., None, None]
    fine = (torch.isfinite(k) | ~live).all(4).all(2)                  # [R, N, Hkv]
    up = torch.where(live, k, -math.inf).amax(2)
    low = torch.where(live, k, math.inf).amin(2)
    scale = _pow2_scale(torch.maximum(up.abs(), low.abs()).amax(-1).nan_to_num(0.0, 0.0, 0.0), _TOPB)
    up = torch.ceil(up / scale[..., None]).clamp(-_TOPB, _TOPB)
    low = torch.floor(low / scale[..., None]).clamp(-_TOPB, _TOPB)
    codes = torch.where(fine[..., None, None], torch.stack((up, low), 3), 0.0).to(torch.int8)
    scale = torch.where(fine, scale, math.inf)
    r, n = touched.nonzero(as_tuple=True)
    s["bounds"][phys[r, n]] = codes[r, n]
    s["bounds_scale"][phys[r, n]] = scale[r, n]
    return s["bounds"], s["bounds_scale"]


def _plain_select(s):
    bounds, q, bs, most = s["bounds"], s["q"], s["block_size"], s["block_lists"].shape[2]
    hkv, d = bounds.shape[1], bounds.shape[3]
    t = s["block_tables"].long().clamp(min=0)
    qf = _grouped(q, hkv)
    qs = _pow2_scale(qf.abs().amax(-1), _TOPB)                        # [B, Hkv, G]
    code = torch.round(qf / qs[..., None]).clamp(-_TOPB, _TOPB)
    both = torch.cat((code.clamp(min=0), code.clamp(max=0)), -1)      # with upper, with lower
    b = bounds[t].float().flatten(3).permute(0, 2, 3, 1)              # [B, Hkv, 2 D, MB]
    bsc = s["bounds_scale"][t].transpose(1, 2)[:, :, None, :]         # [B, Hkv, 1, MB]
    score = torch.where(torch.isinf(bsc), math.inf, (both @ b) * qs[..., None] * bsc)
    score = score.amax(2)                                             # [B, Hkv, MB]
    n = ((s["seq_lens"].long() + bs - 1) // bs)[:, None, None]
    j = torch.arange(t.shape[1], device=q.device)
    # 3: kept whatever the score; 2: a block with a key that is not finite;
    # 1: by score; 0: past the end
    kept = (j < s["sink"]) | (j >= n - s["recent"])
    rank = torch.where(j >= n, 0, torch.where(kept, 3, torch.where(torch.isinf(score), 2, 1)))
    score = torch.where(rank == 1, score, 0.0)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = order.gather(2, torch.sort(rank.expand_as(score).gather(2, order), dim=-1,
                                       descending=True, stable=True).indices)
    k = min(most, t.shape[1])
    count = torch.minimum(n, torch.full_like(n, most))
    chosen = torch.where(torch.arange(k, device=q.device) < count, order[..., :k], 1 << 30)
    chosen = chosen.sort(-1).values
    s["block_lists"].fill_(-1)
    s["block_lists"][..., :k] = torch.where(chosen < 1 << 30, chosen, -1).int()
    s["list_lens"].copy_(count[:, 0, 0])
    return s["block_lists"], s["list_lens"]


def _plain_sparse(s):
    pool, q, bs, lists = s["kv_cache"], s["q"], s["block_size"], s["block_lists"].long()
    b, hkv, k = lists.shape
    d = pool.shape[4]
    here = (lists >= 0) & (torch.arange(k, device=q.device) < s["list_lens"][:, None, None])
    at = lists.clamp(min=0)
    phys = s["block_tables"].long().gather(1, at.flatten(1)).view(b, hkv, k).clamp(min=0)
    head = torch.arange(hkv, device=q.device)[None, :, None]
    kk, vv = pool[0].transpose(1, 2)[phys, head], pool[1].transpose(1, 2)[phys, head]
    if s["kv_scales"] is not None:                                    # [B, Hkv, K, bs, D]
        kk = _value8(kk) * s["kv_scales"][0][phys, head][..., None, None]
        vv = _value8(vv) * s["kv_scales"][1][phys, head][..., None, None]
    p = at[..., None] * bs + torch.arange(bs, device=q.device)
    live = here[..., None] & (p < s["seq_lens"][:, None, None, None])
    o = _attend(_grouped(q, hkv), kk.float().flatten(2, 3), vv.float().flatten(2, 3),
                live.flatten(2, 3), s["scale"])
    return o.view(b, -1, d).to(q.dtype)


# ---------------------------------------------------------------------------
# What a program has in hand, and one pass
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, new = _lens(case)
    nblk = _blocks(case, lens)
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_size"], case["block_size"]
    dtype, b = _DTYPE[case["dtype"]], case["seqs"]
    nb, mb = int(1.25 * sum(nblk)) + 1, max(1, max(nblk))
    n = torch.tensor(nblk, device=dev)
    j = torch.arange(mb, device=dev)[None]
    deal = torch.randperm(nb, generator=g, device=dev)
    at = ((n.cumsum(0) - n)[:, None] + j).clamp(max=nb - 1)
    s = dict(op=case["op"], block_size=bs, scale=1.0 / math.sqrt(d), max_seq_len=max(lens),
             max_query_len=max(new), kv_scales=None,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             new_lens=torch.tensor(new, device=dev),
             block_tables=torch.where(j < n[:, None], deal[at], -1).int().contiguous())
    s["query_start_loc"] = torch.zeros(b + 1, dtype=torch.int32, device=dev)
    s["query_start_loc"][1:] = s["new_lens"].cumsum(0)
    # keys have a few louder channels, as projections of real states do
    loud = torch.exp(0.5 * torch.randn(2, hkv, d, generator=g, device=dev))
    loud[1] = 1.0
    eight = case["op"] in ("write8", "decode8") or case.get("pool") == "8bit"
    if case["op"] != "select":
        s["kv_cache"] = torch.empty(2, nb, bs, hkv, d, device=dev,
                                    dtype=torch.uint8 if eight else dtype)
        if eight:
            s["kv_scales"] = torch.empty(2, nb, hkv, device=dev)
        step = max(1, (1 << 28) // (bs * hkv * d))
        for plane in range(2):
            for i in range(0, nb, step):
                x = torch.randn(min(step, nb - i), bs, hkv, d, generator=g, device=dev)
                x = (x * loud[plane]).to(dtype)
                if eight:
                    x = x.float()
                    sc = _pow2_scale(x.abs().amax((1, 3)), _TOP8)
                    s["kv_scales"][plane, i:i + step] = sc
                    x = _e4m3(x / sc[:, None, :, None])
                s["kv_cache"][plane, i:i + step] = x
    if case["op"] in ("decode8", "select", "sparse"):
        s["q"] = torch.randn(b, h, d, generator=g, device=dev).to(dtype)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "write8":
        for plane, name in enumerate(("key", "value")):
            x = torch.randn(sum(new), hkv, d, generator=g, device=dev)
            s[name] = (x * loud[plane]).to(dtype)
    if case["op"] in ("bounds", "select"):
        s["bounds"] = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device=dev)
        s["bounds_scale"] = torch.ones(nb, hkv, device=dev)
    if case["op"] == "select":  # bounds of blocks of such keys
        step = max(1, (1 << 28) // (bs * hkv * d))
        for i in range(0, nb, step):
            x = torch.randn(min(step, nb - i), bs, hkv, d, generator=g, device=dev)
            x = (x * loud[0]).to(dtype).float()
            up, low = x.amax(1), x.amin(1)
            sc = _pow2_scale(torch.maximum(up, -low).amax(-1), _TOPB)
            s["bounds"][i:i + step, :, 0] = torch.ceil(up / sc[..., None]).to(torch.int8)
            s["bounds"][i:i + step, :, 1] = torch.floor(low / sc[..., None]).to(torch.int8)
            s["bounds_scale"][i:i + step] = sc
        s.update(sink=case["sink"], recent=case["recent"])
    if case["op"] in ("select", "sparse"):
        k = case["select"]
        s["block_lists"] = torch.full((b, hkv, k), -1, dtype=torch.int32, device=dev)
        s["list_lens"] = torch.zeros(b, dtype=torch.int32, device=dev)
    if case["op"] == "sparse":  # distinct blocks, other ones for every head
        r = torch.rand(b, hkv, mb, generator=g, device=dev)
        r = torch.where((j < n[:, None])[:, None], r, 2.0).sort(-1).indices[..., :k]
        m = torch.minimum(n, torch.full_like(n, k))
        r = torch.where(torch.arange(r.shape[2], device=dev) < m[:, None, None], r, 1 << 30)
        r = r.sort(-1).values
        s["block_lists"][..., :r.shape[2]] = torch.where(r < 1 << 30, r, -1).int()
        s["list_lens"].copy_(m)
    # the workspace that such a program allocates once
    s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device=dev)
    return s


def run(state):
    s = state
    if own:
        import paged_kv_cache_136_gb300 as pa
        if s["op"] == "write8":
            pa.pa_reshape_and_cache_fp8_block(
                s["key"], s["value"], s["kv_cache"], s["kv_scales"], s["block_tables"],
                s["seq_lens"], s["query_start_loc"], s["block_size"], s["max_query_len"])
            return s["kv_cache"].view(torch.float8_e4m3fn), s["kv_scales"]
        if s["op"] == "decode8":
            return pa.pa_decode_fp8_block(
                s["out"], s["q"], s["kv_cache"], s["kv_scales"], s["block_tables"],
                s["seq_lens"], s["scale"], s["block_size"], s["max_seq_len"], s["workspace"])
        if s["op"] == "bounds":
            pa.pa_update_block_bounds(
                s["bounds"], s["bounds_scale"], s["kv_cache"], s["block_tables"], s["seq_lens"],
                s["query_start_loc"], s["block_size"], s["max_query_len"],
                kv_scales=s["kv_scales"])
            return s["bounds"], s["bounds_scale"]
        if s["op"] == "select":
            pa.pa_select_blocks(
                s["block_lists"], s["list_lens"], s["q"], s["bounds"], s["bounds_scale"],
                s["block_tables"], s["seq_lens"], s["block_size"], s["max_seq_len"],
                s["workspace"], num_sink_blocks=s["sink"], num_recent_blocks=s["recent"])
            return s["block_lists"], s["list_lens"]
        return pa.pa_decode_sparse(
            s["out"], s["q"], s["kv_cache"], s["block_tables"], s["seq_lens"],
            s["block_lists"], s["list_lens"], s["scale"], s["block_size"], s["workspace"],
            kv_scales=s["kv_scales"])
    if s["op"] == "write8":
        return _plain_write8(s)
    if s["op"] == "decode8":
        return _plain_decode8(s)
    if s["op"] == "bounds":
        return _plain_bounds(s)
    if s["op"] == "select":
        return _plain_select(s)
    return _plain_sparse(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, request by request
# ---------------------------------------------------------------------------
def _two_to(e):
    """2^e in 64 bits, by its bits: a power function may be off in the last."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _scale_of(amax, top):
    """2^e by comparison with the 121 powers there are."""
    powers = _two_to(torch.arange(-60, 61, device=amax.device))
    i = torch.searchsorted(powers * top, amax.double().contiguous())
    return powers[i.clamp(max=120)]


def _nearest8(x):
    """The e4m3 value nearest to x, ties to the even one, held to +-448."""
    x = x.double()
    quantum = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return (torch.round(x / quantum) * quantum).clamp(-448, 448)


def _codes8(u):
    """e4m3 codes to values by the format: sign, 4 exponent bits, 3 of fraction."""
    u = u.to(torch.int64)
    e, f = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * _two_to(e - 7))
    return torch.where(u & 128 != 0, -mag, mag)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lens(case)
    bs, d = case["block_size"], case["head_size"]
    hkv, grp = case["kv_heads"], case["heads"] // case["kv_heads"]
    tables = s["block_tables"].long()
    if case["op"] == "select":
        lists, most = torch.full_like(s["block_lists"], -1), case["select"]
        q = s["q"].double().view(-1, hkv, grp, d)
        qs = _scale_of(q.abs().amax(-1), 127.0)
        code = torch.round(q / qs[..., None]).clamp(-127, 127)
        for b, length in enumerate(lens):
            n = -(-length // bs)
            keys = s["bounds"][tables[b, :n]].double()                # [n, Hkv, 2, D]
            best = torch.maximum(code[b][None] * keys[:, :, None, 0],
                                 code[b][None] * keys[:, :, None, 1]).sum(-1)
            best = best * qs[b] * s["bounds_scale"][tables[b, :n]].double()[..., None]
            best = best.amax(-1)                                      # [n, Hkv]
            best[:case["sink"]] = math.inf
            best[max(0, n - case["recent"]):] = math.inf
            first = torch.sort(best, dim=0, descending=True, stable=True).indices[:most]
            lists[b, :, :len(first)] = first.sort(0).values.t().int()
        return lists, torch.tensor([min(-(-v // bs), most) for v in lens], dtype=torch.int32)
    if case["op"] == "write8":
        value, scales = _codes8(s["kv_cache"]), s["kv_scales"].double()
        at = 0
        for r, (length, q) in enumerate(zip(lens, new)):
            for j in range((length - q) // bs, (length - 1) // bs + 1 if q else 0):
                lo, hi = max(length - q, j * bs), min(length, (j + 1) * bs)
                blk, o = int(tables[r, j]), lo - j * bs
                rows = slice(at + lo - (length - q), at + hi - (length - q))
                for plane, x in enumerate((s["key"], s["value"])):
                    x = x[rows].double()
                    sc = _scale_of(x.abs().amax((0, 2)), 448.0)
                    if o:
                        was = scales[plane, blk]
                        sc = torch.maximum(sc, was)
                        value[plane, blk, :o] = _nearest8(
                            value[plane, blk, :o] * (was / sc)[None, :, None])
                    value[plane, blk, o:o + hi - lo] = _nearest8(x / sc[None, :, None])
                    scales[plane, blk] = sc
            at += q
        return value, scales
    if case["op"] == "bounds":
        scale = s["bounds_scale"].double()
        for r, (length, q) in enumerate(zip(lens, new)):
            first = (length - q) // bs
            blks = tables[r, first:(length - 1) // bs + 1 if q else first]
            k = s["kv_cache"][0][blks]
            if s["kv_scales"] is not None:
                k = _codes8(k) * s["kv_scales"][0][blks].double()[:, None, :, None]
            k = k.double().abs().clone()
            if q and length % bs:
                k[-1, length % bs:] = 0
            scale[blks] = _scale_of(k.amax((1, 3)), 127.0)
        return None, scale
    out = torch.zeros(case["seqs"], hkv, grp, d, dtype=torch.float64, device=tables.device)
    q64 = s["q"].double().view(-1, hkv, grp, d)
    for b, length in enumerate(lens):
        for h in range(hkv):
            j = torch.arange(-(-length // bs), device=tables.device)
            if case["op"] == "sparse":
                j = s["block_lists"][b, h, :int(min(case["select"], len(j)))].long()
            elif h:
                continue
            hs = slice(h, h + 1) if case["op"] == "sparse" else slice(0, hkv)
            blk = tables[b, j]
            kv = s["kv_cache"][:, blk][:, :, :, hs]                   # [2, n, bs, heads, D]
            if s["kv_scales"] is not None:
                kv = _codes8(kv) * s["kv_scales"][:, blk].double()[:, :, None, hs, None]
            live = (j[:, None] * bs + torch.arange(bs, device=j.device) < length).flatten()
            k, v = kv.double().flatten(1, 2)[:, live].unbind(0)       # [L, heads, D]
            a = torch.einsum("hgd,lhd->hgl", q64[b, hs], k) / math.sqrt(d)
            out[b, hs] = torch.einsum("hgl,lhd->hgd", torch.softmax(a, -1), v)
    return out.view(case["seqs"], -1, d)
