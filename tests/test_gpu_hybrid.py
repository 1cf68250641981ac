"""A small server's step, as a program would write it: a softmax layer over a paged
cache and a linear-attention layer over a pool of states, both kept by fork, extend and
compact.  Every step is compared with plain 64-bit sums over each sequence's own
history, which knows nothing of blocks."""
import math

import pytest
import torch

from tests._linear_ref import SLACK

pytestmark = pytest.mark.gpu
I32, BS, ONE = torch.int32, 16, 1 << 24     # ONE: the block size of a pool of states


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    pa.pa_device_errors(clear=True)
    return pa


class Plain:
    """One sequence: its keys and values, its linear layer's sums, and how many calls
    those went through."""

    def __init__(self, hkv, d):
        self.k = torch.zeros(0, hkv, d, dtype=torch.float64)
        self.v = torch.zeros(0, hkv, d, dtype=torch.float64)
        self.S = torch.zeros(hkv, d, d, dtype=torch.float64)
        self.M, self.calls = self.S.clone(), 0

    def copy(self):
        to = Plain(*self.S.shape[:2])
        to.k, to.v, to.S, to.M, to.calls = self.k, self.v, self.S, self.M, self.calls
        return to

    def step(self, q, k, v, g, scale):
        """Rows of both layers, and the sums of absolute values behind them."""
        self.calls += 1
        rows = [[], [], [], []]
        for t in range(len(q)):
            self.k = torch.cat([self.k, k[t:t + 1]])
            self.v = torch.cat([self.v, v[t:t + 1]])
            hkv, d = k.shape[1:]
            qt = q[t].view(hkv, -1, d) * scale
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", qt, self.k), dim=-1)
            kv, a = k[t][:, :, None] * v[t][:, None, :], torch.exp(g[t])[:, None, None]
            self.S, self.M = a * self.S + kv, a * self.M + kv.abs()
            for r, x in zip(rows, (torch.einsum("hgn,nhd->hgd", p, self.v),
                                   torch.einsum("hgn,nhd->hgd", p, self.v.abs()),
                                   qt @ self.S, qt.abs() @ self.M)):
                r.append(x.reshape(-1, d))
        return [torch.stack(r) for r in rows]


class Server:
    def __init__(self, pa, rows, dtype, heads=4, hkv=2, d=64, blocks=60, wide=12, states=14, room=64):
        self.pa, self.rows, self.dt, self.wide = pa, rows, dtype, wide
        self.heads, self.hkv, self.d, self.scale = heads, hkv, d, 1 / math.sqrt(d)
        self.kv = torch.full((2, blocks, BS, hkv, d), float("nan"), dtype=dtype, device="cuda")
        self.states = torch.full((states, hkv, d, d), float("nan"), device="cuda")
        z = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
        # two sets of (tables, lens, refs): one for the pages, one for the states
        self.pages, self.homes = [z(rows, wide), z(rows), z(blocks)], [z(rows, 1), z(rows), z(states)]
        self.new, self.parents, self.starts = z(rows), z(rows), z(rows + 1)
        self.info, self.ids, self.sids = z(4), z(blocks), z(states)
        self.slots = torch.zeros(room, dtype=torch.int64, device="cuda")
        self.sslots = torch.zeros(room, dtype=torch.int64, device="cuda")
        self.ws = torch.zeros(max(pa.pa_sequences_workspace_size(rows, blocks),
                                  pa.pa_linear_prefill_workspace_size(rows, room, room, hkv, d)),
                              dtype=torch.uint8, device="cuda")
        self.x = torch.zeros(room, (heads + 2 * hkv) * d, dtype=dtype, device="cuda")
        self.g = torch.zeros(room, hkv, device="cuda")
        self.out = [torch.full((room, heads, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        self.plain = [Plain(hkv, d) for _ in range(rows)]
        self.gen = torch.Generator().manual_seed(3)

    # ---- the program's calls: nothing here reads the device ----
    def run(self, most):
        """New tokens of every row through both layers; `most` 1: the calls for single
        tokens (row s is token s), else those for prompts."""
        pa, h, hkv, d = self.pa, self.heads, self.hkv, self.d
        fresh = self.pages[1] == 0
        for book, slots, pools, bs, info in (
                (self.pages, self.slots, [self.kv], BS, self.info[:2]),
                (self.homes, self.sslots, [self.states[None]], ONE, self.info[2:])):
            pa.pa_extend_sequences(*book, slots, info, *book, self.new, pools, bs, self.ws)
        n = self.rows if most == 1 else len(self.x)
        q, k, v = self.x[:n].split([h * d, hkv * d, hkv * d], dim=1)
        q, k, v = q.view(n, h, d), k.view(n, hkv, d), v.view(n, hkv, d)
        dst = torch.where(self.new > 0, self.homes[0][:, 0], -1)
        src = torch.where(fresh, -1, dst)
        soft, lin = self.out[0][:n], self.out[1][:n]
        tables, lens, _ = self.pages
        if most == 1:
            # slots come packed; here every row has its token at its own place
            first = torch.cumsum(self.new, 0) - self.new
            slots = torch.where(self.new > 0, self.slots[first], -1)
            pa.pa_reshape_and_cache(k, v, self.kv, slots, BS)
            pa.pa_decode(soft, q.contiguous(), self.kv, tables, lens, self.scale, BS)
            pa.pa_linear_decode(lin, q, k, v, self.g[:n], self.states, src, dst, self.scale)
        else:
            pa.pa_reshape_and_cache(k, v, self.kv, self.slots, BS)
            pa.pa_prefill(soft, q.contiguous(), self.kv, tables, lens, self.starts, self.scale,
                          BS, most)
            pa.pa_linear_prefill(lin, q, k, v, self.g, self.states, src, dst, self.starts,
                                 self.scale, most, self.ws)

    def fork(self):
        for i, bs in ((0, BS), (1, ONE)):
            old = self.pages if i == 0 else self.homes
            to = [torch.zeros_like(t) for t in old]
            self.pa.pa_fork_sequences(*to, *old, self.parents, bs)
            for a, b in zip(old, to):
                a.copy_(b)

    def compact(self):
        for (tables, lens, refs), pools, bs, ids, info in (
                (self.pages, [self.kv], BS, self.ids, self.info[:2]),
                (self.homes, [self.states[None]], ONE, self.sids, self.info[2:])):
            self.pa.pa_compact_blocks(tables, refs, ids, info, tables, lens, refs, pools, bs, self.ws)

    # ---- the test's side ----
    def inputs(self, new):
        t = sum(new)
        x = torch.randn(self.x.shape, generator=self.gen).to(self.dt)
        self.x.copy_(x)
        self.g.copy_(-torch.rand(self.g.shape, generator=self.gen) / 8)
        self.new.copy_(torch.tensor(new, dtype=I32))
        self.starts.copy_(torch.tensor([sum(new[:i]) for i in range(self.rows + 1)], dtype=I32))
        for o in self.out:
            o.fill_(7.0)
        return t

    def check(self, new, rows_of_tokens):
        """`rows_of_tokens[s]`: row s's token rows."""
        h, hkv, d = self.heads, self.hkv, self.d
        x, g = self.x.double().cpu(), self.g.double().cpu()
        q, k, v = x.split([h * d, hkv * d, hkv * d], dim=1)
        half = torch.finfo(self.dt).eps / 2
        soft, lin = (o.double().cpu() for o in self.out)
        home, states = self.homes[0][:, 0].tolist(), self.states.double().cpu()
        for s, n in enumerate(new):
            if n == 0:
                continue
            at, p = rows_of_tokens[s], self.plain[s]
            a, a_mag, b, b_mag = p.step(q[at].view(n, h, d), k[at].view(n, hkv, d),
                                        v[at].view(n, hkv, d), g[at], self.scale)
            # softmax: its weights and its output are rounded to half a step each, the
            # scores and sums are fp32
            err = (soft[at] - a).abs() - half * a.abs() - (half + 2.0 ** -18) * a_mag
            assert float(err.max()) <= 0, (s, "softmax", float(err.max()))
            # every call that the state went through adds at most SLACK of the sums of
            # absolute values, which decay as the errors do
            slack = p.calls * SLACK[self.dt]
            err = (lin[at] - b).abs() - half * b.abs() - (1 + half) * slack * b_mag - 2.0 ** -24
            assert float(err.max()) <= 0, (s, "linear", float(err.max()))
            err = (states[home[s]] - p.S).abs() - slack * p.M - 2.0 ** -24 * p.S.abs()
            assert float(err.max()) <= 0, (s, "state", float(err.max()))

    def books(self):
        """Both sets are what the plain sequences say, and share what they may."""
        for (tables, lens, refs), bs in ((self.pages, BS), (self.homes, ONE)):
            count = [0] * len(refs)
            for row, n, p in zip(tables.tolist(), lens.tolist(), self.plain):
                assert n == len(p.k)
                for b in row[:-(-n // bs)]:
                    count[b] += 1
            assert refs.tolist() == count


def rows_of(new):
    return [slice(sum(new[:i]), sum(new[:i + 1])) for i in range(len(new))]


SINGLE = [slice(i, i + 1) for i in range(64)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_serving(pa, dtype, captured):
    """Prompts, single tokens, samples that fork and part, rows that end and start again,
    a smaller pool, speculated tokens; eager, or every step a graph captured once on one
    workspace."""
    s = Server(pa, 6, dtype)
    steps = {"prompts": lambda: s.run(32), "tokens": lambda: s.run(1), "fork": s.fork,
             "compact": s.compact}
    graphs = {}
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for f in steps.values():            # all rows empty, nothing new
                f()
        torch.cuda.current_stream().wait_stream(side)
        for name, f in steps.items():
            graphs[name] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[name]):
                f()
        assert pa.pa_device_errors(clear=True) == 0

    def do(name, new=None):
        if new is not None:
            s.inputs(new)
        graphs[name].replay() if captured else steps[name]()
        if new is not None:
            s.check(new, rows_of(new) if name == "prompts" else SINGLE)
        s.books()
        assert pa.pa_device_errors(clear=True) == 0

    def fork(parents):
        s.parents.copy_(torch.tensor(parents, dtype=I32))
        s.plain = [s.plain[p].copy() if p >= 0 else Plain(s.hkv, s.d) for p in parents]
        do("fork")

    do("prompts", [32, 0, 5, 0, 16, 0])
    do("prompts", [13, 0, 0, 27, 0, 0])         # a prompt's second chunk, a new one
    do("tokens", [1, 0, 1, 1, 1, 0])
    fork([0, 0, 0, 3, 3, -1])                   # samples; two rows end
    assert s.pages[2].max() == 3 and s.homes[2].max() == 3
    do("tokens", [1, 1, 1, 1, 1, 0])            # they part: blocks and states are copied
    assert s.homes[2].max() == 1
    do("tokens", [1, 1, 1, 1, 0, 0])
    fork([2, 4, 1, -1, 2, 1])                   # rows trade places
    do("prompts", [3, 1, 2, 29, 0, 4])          # speculated tokens beside a prompt
    do("compact")
    live, moved = s.info[:2].tolist()
    assert live == int((s.pages[2] > 0).sum()) and int(s.pages[2][live:].max()) == 0
    assert s.info[2].item() == int((s.homes[2] > 0).sum())
    do("tokens", [1, 1, 1, 1, 1, 1])
    fork([-1, 1, -1, 3, -1, 5])
    do("compact")
    do("tokens", [0, 1, 0, 1, 0, 1])
    do("prompts", [20, 1, 0, 0, 30, 1])


def test_without_room_nothing_moves(pa):
    """A step that finds too few blocks says so and leaves every sequence as it was; the
    step goes on once a row has ended."""
    s = Server(pa, 4, torch.float16, blocks=5, states=4)
    s.inputs([30, 16, 0, 0])
    s.run(32)
    s.check([30, 16, 0, 0], rows_of([30, 16, 0, 0]))
    before = [t.clone() for t in (*s.pages, *s.homes)]
    s.inputs([1, 1, 40, 0])
    s.pa.pa_extend_sequences(*s.pages, s.slots, s.info[:2], *s.pages, s.new, [s.kv], BS, s.ws)
    assert s.info[:2].tolist() == [4, -2] and set(s.slots.tolist()) == {-1}
    assert all(torch.equal(a, b) for a, b in zip(before, (*s.pages, *s.homes)))
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_POOL
    s.parents.copy_(torch.tensor([-1, 1, 2, 3], dtype=I32))
    s.plain[0] = Plain(s.hkv, s.d)
    s.fork()
    s.inputs([0, 1, 40, 0])
    s.run(40)
    s.check([0, 1, 40, 0], rows_of([0, 1, 40, 0]))
    s.books()
    assert pa.pa_device_errors(clear=True) == 0
