"""The operators of a hybrid model's cache: their calls, their plain forms and the
sizes at which they are measured.

A hybrid model keeps pages for its softmax layers and one state for each sequence
of its linear-attention layers; both are blocks of a pool.  Five operators:

  lin_prefill  linear attention with a decay for each head over packed prompts:
               S_t = e^(g_t) S_(t-1) + k_t v_t^T,  o_t = scale q_t S_t
  lin_decode   the same for one token of each sequence
  fork         every row of a new block table becomes a copy of one row of the old
               table, or empty; the blocks' reference counts follow
  extend       room for new tokens: the lowest free blocks in row order, copies of
               last blocks that are shared, and the new tokens' slots
  compact      the live blocks move to the front of the pool, tables follow

States are float32 [num_states, num_kv_heads, head_size, head_size] (key channel,
value channel); log decays are float32, one for each kv head or for each token
and kv head.  A block is free when its reference count is zero.
"""
import math
import random

import torch

own = False

_DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
_CHUNK = 128       # tokens that the plain prompt form takes at once


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _linear(name, op, seqs, lo, hi, heads, kv_heads, head_size, dtype, decay, fresh=0):
    c = dict(op=op, seqs=seqs, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads,
             head_size=head_size, dtype=dtype, decay=decay, fresh=fresh, lens_seed=1)
    if name:
        c["name"] = name
    return c


def _blocks_case(name, op, groups, width, lo, hi, block_size, **more):
    c = dict(op=op, groups=groups, width=width, lo=lo, hi=hi, block_size=block_size, lens_seed=1)
    if name:
        c["name"] = name
    c.update(more)
    return c


def listed():
    return [
        # a chat turn of 100 tokens alone on the card: latency
        _linear("lin_prefill small", "lin_prefill", 1, 100, 100, 4, 4, 64, "fp16", "head", fresh=1),
        # 16 prompts and continued chunks, one kv head for each query head
        _linear("lin_prefill mha 16", "lin_prefill", 16, 256, 2048, 32, 32, 128, "fp16", "head",
                fresh=2),
        # one context of 131072 tokens, grouped queries, decays of each token
        _linear("lin_prefill long", "lin_prefill", 1, 131072, 131072, 64, 8, 128, "bf16", "token",
                fresh=1),
        # a step of four requests of a small model
        _linear("lin_decode tiny", "lin_decode", 4, 1, 1, 4, 4, 64, "fp16", "head"),
        # a step of 64 requests, one kv head for each query head
        _linear("lin_decode mha 64", "lin_decode", 64, 1, 1, 32, 32, 128, "fp16", "head"),
        # a step of 256 requests, grouped queries, decays of each token
        _linear("lin_decode gqa 256", "lin_decode", 256, 1, 1, 32, 8, 128, "bf16", "token"),
        # four requests of four beams each
        _blocks_case("fork small", "fork", 4, 4, 16, 512, 16),
        # 128 requests of four beams over long contexts
        _blocks_case("fork long", "fork", 128, 4, 8192, 65536, 16),
        # a decode step of 256 rows, half of them just forked: one new token each
        _blocks_case("extend step", "extend", 64, 4, 16, 4096, 16, new_lo=1, new_hi=1, layers=2,
                     kv_heads=8, head_size=128),
        # 64 prompts and continued chunks
        _blocks_case("extend prompts", "extend", 64, 1, 0, 4096, 16, new_lo=256, new_hi=2048,
                     layers=1, kv_heads=8, head_size=128),
        # a small pool of which four fifths are in use
        _blocks_case("compact small", "compact", 16, 1, 16, 512, 16, fill=0.8, layers=1,
                     kv_heads=4, head_size=64),
        # a pool of 256 requests of which half has been freed, two layers
        _blocks_case("compact half", "compact", 256, 1, 16, 4096, 16, fill=0.5, layers=2,
                     kv_heads=8, head_size=128),
    ]


_HEADS = [(4, 4), (8, 1), (16, 8), (12, 3), (32, 32), (32, 8), (64, 8), (32, 16), (6, 6), (40, 5)]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_prefill", "lin_decode", "fork", "extend", "compact"])
    if op.startswith("lin"):
        heads, kv_heads = rng.choice(_HEADS)
        d, hi = rng.choice([64, 128, 128]), 1
        seqs = _spread(rng, 1, 256)
        if op == "lin_prefill":
            hi = _spread(rng, 1, 131072)
            # at most the padded rows of the largest listed case
            room = (131072 * 64 * 128) // (hi * heads * d)
            seqs = max(1, min(_spread(rng, 1, 64), room))
        c = _linear("", op, seqs, max(1, hi // 8) if rng.random() < 0.7 else hi, hi, heads,
                    kv_heads, d, rng.choice(["fp16", "bf16"]), rng.choice(["head", "token"]),
                    fresh=rng.choice([0, 1, 2, 3]))
    else:
        width = rng.choice([1, 2, 4, 4, 8])
        hi = _spread(rng, 16, 65536 if op == "fork" else 8192)
        # at most the blocks of the largest listed cases
        room = (512 * 36864 if op == "fork" else 256 * 1024) // (hi * width)
        groups = max(1, min(_spread(rng, 1, 256), room))
        more = {}
        if op != "fork":
            heads, d = rng.choice([(1, 128), (4, 64), (8, 64), (8, 128), (5, 128)])
            more.update(layers=rng.choice([1, 1, 2]), kv_heads=heads, head_size=d)
        if op == "extend":
            more["new_lo"] = rng.choice([0, 1, 1])
            more["new_hi"] = rng.choice([1, 1, max(1, min(_spread(rng, 1, 2048), hi))])
        if op == "compact":
            more["fill"] = rng.choice([0.3, 0.5, 0.7, 0.9])
        c = _blocks_case("", op, groups, width, max(0 if op == "extend" else 1, hi // 16), hi,
                         rng.choice([16, 16, 32]), **more)
    c["lens_seed"] = rng.randrange(1 << 20)
    return c


def _lens(case):
    """Tokens of every sequence (of every group of rows), by the case alone."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "lin_prefill":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["op"] == "extend" and case["new_hi"] > 1:  # every other prompt is a new one
        return [r.randint(case["lo"], case["hi"]) if i % 2 else 0 for i in range(case["groups"])]
    lo, hi = max(1, case["lo"]), case["hi"]
    mid = math.log(max(1.0, hi / 4))
    return [min(hi, max(lo, int(round(math.exp(r.gauss(mid, 1.0)))))) for _ in range(case["groups"])]


def _new(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["groups"] * case["width"])]


def _forked(case, g):
    """Whether the rows of group g share every block (they were just forked), or all
    but the last few."""
    return case["op"] == "extend" and g % 2 == 0


def _distinct(case):
    """(shared blocks, further blocks of each row) of every group."""
    bs, got = case["block_size"], []
    for g, n in enumerate(_lens(case)):
        nb = -(-n // bs)
        shared = nb if _forked(case, g) else min(n // bs, nb - nb // 8)
        got.append((shared, nb - shared))
    return got


def _taken(case):
    """(blocks that an extend takes, last blocks that it copies)."""
    bs, w, new = case["block_size"], case["width"], _new(case)
    taken = copied = 0
    for g, n in enumerate(_lens(case)):
        mine = new[g * w:(g + 1) * w]
        taken += sum(-(-(n + q) // bs) - -(-n // bs) for q in mine)
        if _forked(case, g) and n % bs:
            some = sum(q > 0 for q in mine)
            copied += some - 1 if some == w else some
    return taken + copied, copied


def _num_blocks(case):
    used = sum(a + b * case["width"] for a, b in _distinct(case))
    if case["op"] == "compact":
        return int(used / case["fill"]) + 1
    return int(1.25 * used) + 1 + (_taken(case)[0] if case["op"] == "extend" else 0)


def _page_bytes(case):
    return 4 * case["block_size"] * case["kv_heads"] * case["head_size"] * case["layers"]


def work(case):
    if case["op"].startswith("lin"):
        h, hkv, d = case["heads"], case["kv_heads"], case["head_size"]
        lens = _lens(case) if case["op"] == "lin_prefill" else [1] * case["seqs"]
        t, b = sum(lens), case["seqs"]
        read = b if case["op"] == "lin_decode" else b - sum(_fresh(case, i) for i in range(b))
        decays = hkv * 4 * (t if case["decay"] == "token" else 1)
        # token by token: a state's update 3 D^2 for each kv head, its product 2 D^2 for each head
        return {"bytes": 4 * t * (h + hkv) * d + decays + 4 * (read + b) * hkv * d * d + 12 * b,
                "flops": t * d * d * (3 * hkv + 2 * h)}
    rows, bs = case["groups"] * case["width"], case["block_size"]
    lens = [n for n in _lens(case) for _ in range(case["width"])]
    nb = _num_blocks(case)
    before = sum(-(-n // bs) for n in lens)
    if case["op"] == "fork":
        return {"bytes": 8 * before + 8 * nb + 12 * rows, "flops": before}
    if case["op"] == "extend":
        new = _new(case)
        after = sum(-(-(n + q) // bs) for n, q in zip(lens, new))
        return {"bytes": 4 * (before + after) + 8 * nb + 8 * sum(new) + 16 * rows +
                2 * _taken(case)[1] * _page_bytes(case), "flops": nb + after}
    moved = case["fill"] * (1 - case["fill"]) * nb  # of blocks that lie anywhere
    return {"bytes": 8 * before + 12 * nb + 4 * rows + 2 * moved * _page_bytes(case),
            "flops": nb + before}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_prefill(s):
    q, k, v, g = s["q"], s["k"], s["v"], s["log_decay"]
    h, d, hkv, c = q.shape[1], q.shape[2], k.shape[1], _CHUNK
    start = s["query_start_loc"].long()
    b, n = start.numel() - 1, -(-s["max_query_len"] // c)
    at = start[:-1, None] + torch.arange(n * c, device=q.device)
    live = at < start[1:, None]                                       # [B, N C]
    at = at.clamp(max=q.shape[0] - 1)
    chunks = lambda x: x.view(b, n, c, *x.shape[2:])                  # noqa: E731
    qf = chunks(q[at].float().view(b, n * c, hkv, h // hkv, d))
    kf = chunks(torch.where(live[..., None, None], k[at].float(), 0.0))
    vf = chunks(torch.where(live[..., None, None], v[at].float(), 0.0))
    gt = g[at] if g.dim() == 2 else g.expand(b, n * c, hkv)
    gt = chunks(torch.where(live[..., None], gt.double(), 0.0))
    cum = gt.cumsum(2)                                                # [B, N, C, Hkv]
    total = cum[:, :, -1]                                             # [B, N, Hkv]
    lower = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    by_head = cum.transpose(2, 3)
    decay = torch.where(lower, by_head[..., :, None] - by_head[..., None, :], -math.inf)
    decay = decay.exp().float()                                       # [B, N, Hkv, C, C]
    tail = (total[:, :, None] - cum).exp().float()
    added = torch.einsum("bnchd,bnche->bhnde", kf * tail[..., None], vf)
    # the state before every chunk, and behind the last: all earlier chunks' parts
    ends = torch.cat((torch.zeros_like(total[:, :1]), total), 1).cumsum(1).transpose(1, 2)
    earlier = torch.arange(n + 1, device=q.device)[:, None] > torch.arange(n, device=q.device)
    weight = torch.where(earlier, ends[..., :, None] - ends[..., None, 1:], -math.inf)
    src = s["src_states"].long()
    first = torch.where((src >= 0)[:, None, None, None], s["states"][src.clamp(min=0)], 0.0)
    before = weight.exp().float() @ added.flatten(3)                  # [B, Hkv, N + 1, D D]
    before += ends.exp().float()[..., None] * first.flatten(2)[:, :, None]
    before = before.view(b, hkv, n + 1, d, d)
    o = torch.einsum("bnchgd,bhnde->bnchge", qf, before[:, :, :n])
    o *= cum.exp().float()[..., None, None]
    p = torch.einsum("bnchgd,bnjhd->bnhgcj", qf, kf) * decay[:, :, :, None]
    o += torch.einsum("bnhgcj,bnjhe->bnchge", p, vf)
    s["states"][s["dst_states"].long()] = before[:, :, n]
    s["out"][at[live]] = (o * s["scale"]).reshape(b, n * c, h, d)[live].to(q.dtype)
    return s["out"], s["states"]


def _plain_decode(s):
    q, k, v = s["q"], s["k"].float(), s["v"].float()
    b, h, d = q.shape
    hkv = k.shape[1]
    src = s["src_states"].long()
    state = torch.where((src >= 0)[:, None, None, None], s["states"][src.clamp(min=0)], 0.0)
    state = s["log_decay"].exp().expand(b, hkv)[..., None, None] * state
    state = state + k[..., :, None] * v[..., None, :]
    s["states"][s["dst_states"].long()] = state
    o = q.float().view(b, hkv, h // hkv, d) @ state * s["scale"]
    s["out"].copy_(o.view(b, h, d))
    return s["out"], s["states"]


def _used(tables, seq_lens, bs):
    """Which entries of the tables hold a block."""
    n = (seq_lens.long() + bs - 1) // bs
    return torch.arange(tables.shape[1], device=tables.device) < n[:, None]


def _plain_fork(s):
    tables, lens, bs = s["block_tables"], s["seq_lens"], s["block_size"]
    parents = s["parents"].long()
    here = parents >= 0
    of = parents.clamp(min=0)
    new_lens = torch.where(here, lens[of], 0)
    s["seq_lens_out"].copy_(new_lens)
    s["tables_out"].copy_(torch.where(_used(tables, new_lens, bs), tables[of], s["tables_out"]))
    children = torch.zeros_like(lens).index_add_(0, of, here.to(torch.int32))
    used = _used(tables, lens, bs)
    delta = (children - 1)[:, None].expand_as(tables)[used]
    s["ref_counts_out"].copy_(s["ref_counts"])
    s["ref_counts_out"].index_add_(0, tables[used].long(), delta)
    return s["tables_out"], s["seq_lens_out"], s["ref_counts_out"]


def _plain_extend(s):
    tables, lens, refs = s["block_tables"], s["seq_lens"].long(), s["ref_counts"]
    new, bs, dev = s["num_new"].long(), s["block_size"], s["seq_lens"].device
    rows, wide, nb = tables.shape[0], tables.shape[1], refs.numel()
    row = torch.arange(rows, device=dev)
    before, after = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
    # a row that writes into a shared last block copies it; where all holders of the
    # block write, the last of them keeps it
    last = tables.long().gather(1, (before - 1).clamp(min=0)[:, None])[:, 0]
    writes = (new > 0) & (lens % bs != 0)
    at = torch.where(writes, last, nb)
    writers = torch.zeros(nb + 1, dtype=torch.long, device=dev).index_add_(
        0, at, torch.ones_like(at))
    latest = torch.full((nb + 1,), -1, dtype=torch.long, device=dev).scatter_reduce_(
        0, at, row, "amax")
    count = refs.long()[last.clamp(min=0, max=nb - 1)]
    keeps = (writers[at] == count) & (latest[at] == row)
    copies = writes & (count > 1) & ~keeps
    need = after - before + copies
    begin = need.cumsum(0) - need
    free = (refs == 0).nonzero()[:, 0]
    s["info"][0] = need.sum()
    s["info"][1] = free.numel() - need.sum()
    j = torch.arange(wide, device=dev)
    fresh = ((j >= before[:, None]) & (j < after[:, None])) | \
        (copies[:, None] & (j == (before - 1)[:, None]))
    rank = begin[:, None] + j - before[:, None] + copies[:, None]
    got = torch.where(fresh, free[rank.clamp(0, max(0, free.numel() - 1))].int(), tables)
    s["tables_out"].copy_(torch.where(j < after[:, None], got, s["tables_out"]))
    s["seq_lens_out"].copy_(lens + new)
    out = s["ref_counts_out"]
    out.copy_(refs)
    out[free[:int(need.sum())]] = 1
    out.index_add_(0, last[copies], torch.full_like(last[copies], -1, dtype=torch.int32))
    end = new.cumsum(0)
    t = torch.arange(s["slot_mapping"].numel(), device=dev)
    of = torch.searchsorted(end, t, right=True)
    of_row = of.clamp(max=rows - 1)
    p = (lens + new - end)[of_row] + t
    block = s["tables_out"].long()[of_row, (p // bs).clamp(max=wide - 1)]
    s["slot_mapping"].copy_(torch.where(of < rows, block * bs + p % bs, -1))
    for pool in s["pools"]:
        pool[:, free[begin[copies]]] = pool[:, last[copies]]
    return (s["tables_out"], s["seq_lens_out"], out, s["slot_mapping"], s["info"], s["pools"])


def _plain_compact(s):
    tables, refs, bs = s["block_tables"], s["ref_counts"], s["block_size"]
    live = refs > 0
    n = live.sum()
    place = torch.arange(refs.numel(), device=refs.device)
    src, dst = (live & (place >= n)).nonzero()[:, 0], (~live & (place < n)).nonzero()[:, 0]
    new = torch.where(live, place, -1).int()
    new[src] = dst.int()
    s["new_ids"].copy_(new)
    s["info"][0] = n
    s["info"][1] = src.numel()
    s["ref_counts_out"].copy_(refs)
    s["ref_counts_out"][dst] = refs[src]
    s["ref_counts_out"][src] = 0
    used = _used(tables, s["seq_lens"], bs)
    s["tables_out"].copy_(torch.where(used, new[tables.long().clamp(min=0)], s["tables_out"]))
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]
    return s["tables_out"], s["ref_counts_out"], s["new_ids"], s["info"], s["pools"]


# ---------------------------------------------------------------------------
# What a program has in hand, and one pass
# ---------------------------------------------------------------------------
def _fresh(case, i):
    """Whether prompt i starts from nothing: all, every second, third, ... or none."""
    return bool(case["fresh"]) and i % case["fresh"] == 0


def _prepare_linear(case, gen, dev):
    h, hkv, d, b = case["heads"], case["kv_heads"], case["head_size"], case["seqs"]
    dtype = _DTYPE[case["dtype"]]
    lens = _lens(case) if case["op"] == "lin_prefill" else [1] * b
    t = sum(lens)
    randn = lambda *n: torch.randn(*n, generator=gen, device=dev)     # noqa: E731
    s = dict(op=case["op"], scale=1.0 / math.sqrt(d), max_query_len=max(lens),
             q=randn(t, h, d).to(dtype), k=randn(t, hkv, d).to(dtype), v=randn(t, hkv, d).to(dtype))
    # a head forgets within some tokens, another one within hundreds
    rate = -torch.exp2(-8.0 * (torch.arange(hkv, device=dev) + 1) / hkv)
    s["log_decay"] = rate.float()
    if case["decay"] == "token":
        s["log_decay"] = (rate * 2 * torch.rand(t, hkv, generator=gen, device=dev)).contiguous()
    # the next states go elsewhere, so that a step can be taken back
    s["states"] = 4 * randn(2 * b, hkv, d, d)
    deal = torch.randperm(2 * b, generator=gen, device=dev).int()
    s["src_states"], s["dst_states"] = deal[:b].clone(), deal[b:].clone()
    if case["op"] == "lin_prefill":
        s["src_states"][torch.tensor([_fresh(case, i) for i in range(b)], device=dev)] = -1
        s["query_start_loc"] = torch.zeros(b + 1, dtype=torch.int32, device=dev)
        s["query_start_loc"][1:] = torch.tensor(lens, device=dev).cumsum(0)
    s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_blocks(case, gen, dev):
    bs, w, nb = case["block_size"], case["width"], _num_blocks(case)
    lens, rows = _lens(case), case["groups"] * case["width"]
    new = _new(case) if case["op"] == "extend" else [0] * rows
    wide = max(1, max(-(-(lens[i // w] + q) // bs) for i, q in enumerate(new)))
    # ids in order of groups, dealt over the pool
    shared, base, more, at = [], [], [], 0
    for a, c in _distinct(case):
        for i in range(w):
            shared.append(a)
            base.append(at)
            more.append(at + i * c)
        at += a + w * c
    put = lambda x, kind=torch.int64: torch.tensor(x, dtype=kind, device=dev)  # noqa: E731
    j = torch.arange(wide, device=dev)
    deal = torch.randperm(nb, generator=gen, device=dev)
    ids = torch.where(j < put(shared)[:, None], put(base)[:, None], put(more)[:, None]) + j
    s = dict(op=case["op"], block_size=bs, max_blocks=wide,
             seq_lens=put([n for n in lens for _ in range(w)], torch.int32))
    used = _used(ids, s["seq_lens"], bs)
    s["block_tables"] = torch.where(used, deal[ids.clamp(max=nb - 1)], -1).int().contiguous()
    s["ref_counts"] = torch.bincount(s["block_tables"][used], minlength=nb).int()
    s["tables_out"] = torch.full_like(s["block_tables"], -1)
    s["ref_counts_out"] = torch.empty_like(s["ref_counts"])
    s["seq_lens_out"] = torch.empty_like(s["seq_lens"])
    if case["op"] == "fork":  # each beam continues one of its request's beams; some requests end
        beam = torch.randint(0, w, (rows,), generator=gen, device=dev)
        parents = torch.arange(rows, device=dev) // w * w + beam
        done = torch.rand(case["groups"], generator=gen, device=dev) < 0.1
        s["parents"] = torch.where(done.repeat_interleave(w), -1, parents).int()
    if case["op"] == "extend":
        s["num_new"] = put(new, torch.int32)
        s["slot_mapping"] = torch.empty(max(1, sum(new)), dtype=torch.int64, device=dev)
    if case["op"] == "compact":
        s["new_ids"] = torch.empty(nb, dtype=torch.int32, device=dev)
    if case["op"] != "fork":
        s["info"] = torch.zeros(2, dtype=torch.int32, device=dev)
        s["pools"] = []
        for _ in range(case["layers"]):
            pool = torch.empty(2, nb, bs, case["kv_heads"], case["head_size"], device=dev,
                               dtype=torch.bfloat16)
            for plane in pool:
                plane.normal_(generator=gen)
            s["pools"].append(pool.view(torch.int16))  # blocks move as they are
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = _prepare_linear if case["op"].startswith("lin") else _prepare_blocks
    s = make(case, gen, "cuda")
    # the workspace that such a program allocates once
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    return s


def run(state):
    s = state
    if own:
        import paged_kv_cache_136_gb300 as pa
        if s["op"] == "lin_prefill":
            pa.pa_linear_prefill(
                s["out"], s["q"], s["k"], s["v"], s["log_decay"], s["states"], s["src_states"],
                s["dst_states"], s["query_start_loc"], s["scale"], s["max_query_len"],
                s["workspace"])
            return s["out"], s["states"]
        if s["op"] == "lin_decode":
            pa.pa_linear_decode(
                s["out"], s["q"], s["k"], s["v"], s["log_decay"], s["states"], s["src_states"],
                s["dst_states"], s["scale"])
            return s["out"], s["states"]
        if s["op"] == "fork":
            pa.pa_fork_sequences(
                s["tables_out"], s["seq_lens_out"], s["ref_counts_out"], s["block_tables"],
                s["seq_lens"], s["ref_counts"], s["parents"], s["block_size"])
            return s["tables_out"], s["seq_lens_out"], s["ref_counts_out"]
        if s["op"] == "extend":
            pa.pa_extend_sequences(
                s["tables_out"], s["seq_lens_out"], s["ref_counts_out"], s["slot_mapping"],
                s["info"], s["block_tables"], s["seq_lens"], s["ref_counts"], s["num_new"],
                s["pools"], s["block_size"], s["workspace"])
            return (s["tables_out"], s["seq_lens_out"], s["ref_counts_out"], s["slot_mapping"],
                    s["info"], s["pools"])
        pa.pa_compact_blocks(
            s["tables_out"], s["ref_counts_out"], s["new_ids"], s["info"], s["block_tables"],
            s["seq_lens"], s["ref_counts"], s["pools"], s["block_size"], s["workspace"])
        return s["tables_out"], s["ref_counts_out"], s["new_ids"], s["info"], s["pools"]
    if s["op"] == "lin_prefill":
        return _plain_prefill(s)
    if s["op"] == "lin_decode":
        return _plain_decode(s)
    if s["op"] == "fork":
        return _plain_fork(s)
    if s["op"] == "extend":
        return _plain_extend(s)
    return _plain_compact(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, token by token
# ---------------------------------------------------------------------------
def exact(case, seed):
    """Outputs and states of the linear operators; the others move whole numbers."""
    if not case["op"].startswith("lin"):
        return None
    h, hkv, d, b = case["heads"], case["kv_heads"], case["head_size"], case["seqs"]
    lens = _lens(case) if case["op"] == "lin_prefill" else [1] * b
    if max(lens) * (1e-4 + 2e-11 * b * hkv * d * d) > 20:
        return None
    s = prepare(case, seed)
    dev = s["q"].device
    order = sorted(range(b), key=lambda i: -lens[i])          # the longest first
    begin = torch.tensor([sum(lens[:i]) for i in order], device=dev)
    by = torch.tensor(order, device=dev)
    src = s["src_states"].long()[by]
    state = s["states"].double()[src.clamp(min=0)]
    state[src < 0] = 0
    factor = torch.exp(s["log_decay"].double())
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    m = b
    for t in range(max(lens)):
        while lens[order[m - 1]] <= t:                        # sequences that have ended
            m -= 1
        at = begin[:m] + t
        a = (factor[at] if factor.dim() == 2 else factor.expand(m, hkv))[..., None, None]
        state[:m] *= a
        state[:m] += s["k"][at].double()[..., None] * s["v"][at].double()[..., None, :]
        o = s["q"][at].double().view(m, hkv, h // hkv, d) @ state[:m]
        out[at] = o.view(m, h, d) / math.sqrt(d)
    states = s["states"].double()
    states[s["dst_states"].long()[by]] = state
    return out, states
