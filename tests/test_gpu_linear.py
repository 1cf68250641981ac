"""Linear attention with a decay for each head on the GPU, against the 64-bit
recurrence of tests/_linear_ref.py."""
import math
import threading

import pytest
import torch

from tests._linear_ref import check_out, check_states, inputs, ref_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    pa.pa_device_errors(clear=True)
    return pa


def decode(pa, x, out=None, stream=None):
    out = torch.full_like(x["q"], 7.0, memory_format=torch.contiguous_format) if out is None else out
    return pa.pa_linear_decode(out, x["q"], x["k"], x["v"], x["log_decay"], x["states"], x["src"],
                               x["dst"], x["scale"], stream=stream)


def longest(x):
    return int((x["starts"][1:] - x["starts"][:-1]).max()) if len(x["starts"]) > 1 else 0


def workspace(pa, x, most=None):
    n = pa.pa_linear_prefill_workspace_size(len(x["src"]), len(x["q"]),
                                            longest(x) if most is None else most,
                                            x["k"].shape[1], x["q"].shape[2])
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def prefill(pa, x, out=None, most=None, ws=None, stream=None):
    out = torch.full_like(x["q"], 7.0, memory_format=torch.contiguous_format) if out is None else out
    most = longest(x) if most is None else most
    return pa.pa_linear_prefill(out, x["q"], x["k"], x["v"], x["log_decay"], x["states"], x["src"],
                                x["dst"], x["starts"], x["scale"], most,
                                workspace(pa, x, most) if ws is None else ws, stream=stream)


def check(pa, x, run, flags=0):
    ref, states, mag, smag = ref_linear(x["q"], x["k"], x["v"], x["log_decay"], x["states"],
                                        x["src"], x["dst"], x["starts"], x["scale"])
    before = x["states"].clone()
    out = run(pa, x)
    check_out(out, ref, mag)
    check_states(x["states"], states, smag, out.dtype)
    assert bool((out[torch.isnan(mag)] == 7.0).all()), "rows that are nobody's were written"
    wrote = torch.zeros(len(before), dtype=torch.bool, device=before.device)
    wrote[[int(i) for i in x["dst"] if 0 <= int(i) < len(before)]] = True
    assert torch.equal(x["states"][~wrote], before[~wrote]), "states that are nobody's were written"
    assert pa.pa_device_errors(clear=True) == flags
    return out


HEADS = [(4, 4), (8, 1), (12, 3), (10, 2), (5, 5), (16, 1)]


@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode(pa, heads, kv_heads, d, dtype):
    for b, decay, fused in ((1, "head", False), (5, "token", True), (37, "token", False)):
        x = inputs([1] * b, heads, kv_heads, d, dtype, decay, seed=b, fresh=range(0, b, 3), fused=fused)
        check(pa, x, decode)


LENS = [[1], [100], [128], [129, 0, 1, 127, 2, 256, 0], [300, 5], [1, 1, 1], [700]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (6, 2), (8, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill(pa, lens, heads, kv_heads, d, dtype):
    for decay, fused in (("head", False), ("token", True)):
        x = inputs(lens, heads, kv_heads, d, dtype, decay, seed=len(lens), fresh=range(1, len(lens), 2),
                   fused=fused, tail=3)
        check(pa, x, prefill)


@pytest.mark.parametrize("lens", [[3000], [513, 0, 1500, 1, 2049, 40], [1024, 1025, 1537]], ids=str)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_in_segments(pa, lens, heads, kv_heads, d, dtype):
    """Few chains that are long: sequences are cut, their segments' states joined."""
    assert pa.pa_linear_prefill_workspace_size(len(lens), sum(lens) + 3, max(lens), kv_heads, d) > 256
    for decay, fresh in (("head", ()), ("token", (0, 2, 5))):
        x = inputs(lens, heads, kv_heads, d, dtype, decay, seed=len(lens), fresh=fresh, tail=3)
        if decay == "head" and len(lens) > 1:
            x["dst"][-1] = -1
        check(pa, x, prefill)


def test_bad_metadata_in_segments(pa):
    """Sequences that overlap or break their bounds are flagged or read twice; no call
    reads or writes outside its tensors."""
    for starts in ([0, 3000, 100, 4000], [0, 4000, 0, 4000, 0, 4000], [-5, 100, 2000, 9000],
                   [0, 1 << 30, 100, 300]):
        x = inputs([4000 // (len(starts) - 1)] * (len(starts) - 1), 2, 1, 64, "fp16", "token", seed=1,
                   tail=4000 % (len(starts) - 1))
        x["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        prefill(pa, x, most=4000)
        assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_not_finite_in_segments(pa, dtype):
    """A value that is not finite reaches the segments behind its own."""
    x = inputs([2000], 2, 2, 64, dtype, "token", seed=2)
    clean = {**x, "states": x["states"].clone()}
    good = prefill(pa, clean)
    x["v"][700, 1, 9] = math.nan
    out = prefill(pa, x)
    keep = torch.arange(64, device="cuda") != 9
    assert torch.equal(out[:700], good[:700]) and torch.equal(out[:, 0], good[:, 0])
    assert torch.equal(out[..., keep], good[..., keep])
    assert bool(torch.isnan(out[700:, 1, 9]).all())
    to = int(x["dst"][0])
    assert bool(torch.isnan(x["states"][to, 1, :, 9]).all())
    assert torch.equal(x["states"][to, 1][:, keep], clean["states"][to, 1][:, keep])
    pa.pa_device_errors(clear=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_equals_decode_steps(pa, d, dtype):
    """A prompt in one call, in two chunks, and token by token: the same states and
    outputs within the bounds of one call each."""
    n = 150
    x = inputs([n], 4, 2, d, dtype, "token", seed=3)
    ref, states, mag, smag = ref_linear(x["q"], x["k"], x["v"], x["log_decay"], x["states"],
                                        x["src"], x["dst"], x["starts"], x["scale"])
    out = torch.empty_like(x["q"])
    cut = 70
    for lo, hi in [(0, cut), (cut, n)]:
        y = {**x, **{key: x[key][lo:hi] for key in ("q", "k", "v", "log_decay")}}
        y["starts"] = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        y["src"] = x["src"] if lo == 0 else x["dst"]
        prefill(pa, y, out=out[lo:hi])
    check_out(out, ref, mag)
    check_states(x["states"], states, smag, out.dtype)
    x = inputs([n], 4, 2, d, dtype, "token", seed=3)
    out.zero_()
    for i in range(n):
        y = {**x, **{key: x[key][i:i + 1] for key in ("q", "k", "v", "log_decay")}}
        y["src"] = x["src"] if i == 0 else x["dst"]
        decode(pa, y, out=out[i:i + 1])
    check_out(out, ref, mag)
    check_states(x["states"], states, smag, out.dtype)


@pytest.mark.parametrize("run", [decode, prefill])
def test_padding_and_bad_ids(pa, run):
    lens = [1] * 6 if run is decode else [130, 3, 140, 0, 9, 1]
    x = inputs(lens, 4, 2, 64, "bf16", "token", seed=5)
    x["dst"][1] = -1                       # a padding row
    x["dst"][2] = -(1 << 31)
    x["src"][4] = -(1 << 31)               # zeros
    check(pa, x, run)
    y = inputs(lens, 4, 2, 64, "bf16", "token", seed=6)
    y["src"][0] = len(y["states"])         # read as zeros
    y["dst"][5] = (1 << 31) - 1            # not written
    check(pa, y, run, flags=pa.DEVERR_STATE)


def test_in_place(pa):
    """src and dst the same: a step of a running batch."""
    for run, lens in ((decode, [1] * 4), (prefill, [129, 1, 0, 260])):
        x = inputs(lens, 8, 2, 128, "fp16", "head", seed=8)
        x["dst"] = x["src"].clone()
        check(pa, x, run)


@pytest.mark.parametrize("run", [decode, prefill])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decays_at_both_ends(pa, run, dtype):
    """Decays of one (0), of zero (-inf and very negative), between ordinary ones."""
    lens = [1] * 12 if run is decode else [5, 260, 131]
    x = inputs(lens, 4, 4, 64, dtype, "token", seed=9)
    g = x["log_decay"]
    pick = torch.rand(g.shape, generator=torch.Generator().manual_seed(1)).cuda()
    g[pick < 0.3] = 0.0
    g[pick > 0.9] = -1e4
    g[pick > 0.95] = -math.inf
    g[pick > 0.98] = -90.0
    check(pa, x, run)


def test_prefill_of_long_memory(pa):
    """Decays of exactly one: the state is a plain sum over all tokens."""
    x = inputs([513], 2, 1, 128, "bf16", "head", seed=10)
    x["log_decay"].zero_()
    check(pa, x, prefill)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_not_finite_stays_where_it_belongs(pa, dtype):
    """NaN and infinities of a token reach that token's row and later ones of its
    sequence, nothing before it, no neighbour, and no rows behind the last."""
    lens = [140, 200, 60]
    for which, value in (("v", math.inf), ("v", math.nan), ("k", math.nan), ("q", math.nan),
                         ("log_decay", math.nan)):
        x = inputs(lens, 4, 2, 64, dtype, "token", seed=11, fresh=(0, 1, 2), tail=70)
        for name in ("q", "k", "v", "log_decay"):
            x[name][sum(lens):] = math.nan
        clean = {**x, "states": x["states"].clone()}
        good = prefill(pa, clean)
        hit = 140 + 150                    # token 150 of sequence 1
        if which == "log_decay":
            x[which][hit, 1] = value
        else:
            x[which][hit, 1, 5] = value
        out = prefill(pa, x)
        rows = torch.ones(len(out), dtype=torch.bool, device="cuda")
        rows[hit:340] = False
        assert torch.equal(out[rows], good[rows]), which
        later = out[hit:340]
        if which == "q":                   # that row's head alone
            assert bool(torch.isnan(out[hit, 1]).all())
            later = later[1:]
            assert torch.equal(later, good[hit + 1:340])
            assert torch.equal(x["states"], clean["states"])
            continue
        # kv head 1 serves query heads 2 and 3; kv head 0 is untouched
        assert torch.equal(later[:, :2], good[hit:340, :2]), which
        if which == "v":                   # value channel 5 alone
            assert not torch.isfinite(later[:, 2:, 5]).any()
            keep = torch.arange(64, device="cuda") != 5
            assert torch.equal(later[:, 2:][..., keep], good[hit:340, 2:][..., keep])
        else:
            assert torch.isnan(later[:, 2:]).all(), which
        S, good_S = x["states"][int(x["dst"][1])], clean["states"][int(x["dst"][1])]
        assert torch.equal(S[0], good_S[0])
        hurt = ~torch.isfinite(S[1])
        if which == "v":
            assert bool(hurt[:, 5].all()) and int(hurt.sum()) == 64
        elif which == "k":
            assert bool(hurt[5].all()) and int(hurt.sum()) == 64
        else:
            assert bool(hurt.all())
        pa.pa_device_errors(clear=True)


def test_prefill_skips_bad_sequences(pa):
    x = inputs([40, 30, 20], 2, 2, 64, "fp16", "head", seed=12)
    want = {**x, "states": x["states"].clone()}
    good = prefill(pa, want)
    out = prefill(pa, x, most=35)          # sequence 0 is longer than max_query_len
    assert torch.equal(out[40:], good[40:]) and bool((out[:40] == 7.0).all())
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    x["starts"] = torch.tensor([0, 40, 30, 95], dtype=torch.int32, device="cuda")
    prefill(pa, x, most=100)               # a negative length, and rows past the end
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN


@pytest.mark.parametrize("scale", [1.0, 3e-4, 40.0])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sizes_of_values(pa, dtype, scale):
    """Loud and quiet keys and values: what leaves fp16's range on the way (scores,
    states) must not leave it in the operands."""
    for lens, run in (([200, 70], prefill), ([1] * 5, decode)):
        x = inputs(lens, 4, 2, 128, dtype, "token", seed=13)
        x["k"] *= scale
        x["q"] *= scale
        x["states"] *= scale
        if scale > 1:
            x["v"] *= 1e-3
        check(pa, x, run)


def test_capture_and_replay(pa):
    """Both calls in one graph; lengths, ids and inputs change between replays."""
    x = inputs([200, 56], 4, 2, 64, "bf16", "token", seed=14)
    y = inputs([1] * 3, 4, 2, 64, "bf16", "token", seed=15)
    out, dec = torch.full_like(x["q"], 7.0), torch.full_like(y["q"], 7.0)
    ws = workspace(pa, x, 256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        prefill(pa, x, out=out, most=256, ws=ws)
        decode(pa, y, out=dec)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prefill(pa, x, out=out, most=256, ws=ws)
        decode(pa, y, out=dec)
    for seed, lens in ((20, [1, 255]), (21, [130, 126])):
        nx, ny = (inputs(a, 4, 2, 64, "bf16", "token", seed=seed) for a in (lens, [1] * 3))
        for old, new in ((x, nx), (y, ny)):
            for key in old:
                if isinstance(old[key], torch.Tensor):
                    old[key].copy_(new[key])
        rx = ref_linear(*(x[k] for k in ("q", "k", "v", "log_decay", "states", "src", "dst",
                                         "starts", "scale")))
        ry = ref_linear(*(y[k] for k in ("q", "k", "v", "log_decay", "states", "src", "dst",
                                         "starts", "scale")))
        g.replay()
        torch.cuda.synchronize()
        check_out(out, rx[0], rx[2])
        check_states(x["states"], rx[1], rx[3], out.dtype)
        check_out(dec, ry[0], ry[2])
        check_states(y["states"], ry[1], ry[3], out.dtype)
    assert pa.pa_device_errors(clear=True) == 0


def test_repeatable_and_on_streams(pa):
    """The same bits every time, on two streams at once with a workspace each."""
    lens = [400, 31, 260]
    xs = [inputs(lens, 8, 2, 128, "bf16", "token", seed=16) for _ in range(3)]
    outs = [torch.full_like(x["q"], 7.0) for x in xs]
    wss = [workspace(pa, x) for x in xs]
    prefill(pa, xs[0], out=outs[0], ws=wss[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, s in enumerate(streams):
        prefill(pa, xs[i + 1], out=outs[i + 1], ws=wss[i + 1], stream=s)
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(outs[i], outs[0]) and torch.equal(xs[i]["states"], xs[0]["states"])


def test_no_sequences_and_no_tokens(pa):
    x = inputs([0, 0], 2, 2, 64, "fp16", "head", seed=17, fresh=(1,))
    check(pa, x, prefill)
    y = inputs([], 2, 2, 64, "fp16", "head", seed=18, tail=4)
    out = prefill(pa, y)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("run", [decode, prefill])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_a_decay_of_zero_forgets_large_states(pa, run, dtype):
    """exp(-inf) is 0, not a small number: nothing of 1e35 is left.  (2^-8 of the sum of
    absolute values is twice the outputs' rounding; the smallest 32-bit number times 1e35
    would be 1e-4 at least, and times the sums of 64 channels more.)"""
    lens = [1] * 3 if run is decode else [5, 1, 300]
    x = inputs(lens, 4, 2, 64, dtype, "token", seed=21)
    x["states"] *= 1e35 / 16
    x["log_decay"][x["starts"][:-1].long()] = -math.inf
    ref, states, mag, smag = ref_linear(*(x[k] for k in ("q", "k", "v", "log_decay", "states", "src",
                                                         "dst", "starts", "scale")))
    out = run(pa, x)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * mag + 2.0 ** -24).all())
    to = x["dst"].long()
    assert bool(((x["states"].double() - states).abs() <= 2.0 ** -15 * smag)[to].all())
    assert pa.pa_device_errors(clear=True) == 0


def test_far_tokens(pa):
    """Token rows, outputs and states beyond 2^32 bytes and 2^31 elements."""
    t, h, hkv, d = 70_000, 256, 2, 128
    # sequences of t - 280 (a padding row), 130, 9 and 141 tokens
    g = torch.Generator().manual_seed(22)
    q = torch.empty(t, h, d, dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    k, v = (torch.randn(t, hkv, d, generator=g).half().cuda() for _ in range(2))
    q[-280:] = torch.randn(280, h, d, generator=g).half().cuda()
    out[-280:], out[:9] = 7.0, 7.0
    decay = (-torch.rand(t, hkv, generator=g) / 16).cuda()
    ns = (1 << 31) // (hkv * d * d) + 8
    states = torch.empty(ns, hkv, d, d, device="cuda")
    src = torch.tensor([3, ns - 1, -1, ns - 2], dtype=torch.int32, device="cuda")
    dst = torch.tensor([-1, ns - 3, ns - 4, ns - 2], dtype=torch.int32, device="cuda")
    states[-4:] = torch.randn(4, hkv, d, d, generator=g).cuda()
    starts = torch.tensor([0, t - 280, t - 150, t - 141, t], dtype=torch.int32, device="cuda")
    # states[-4:] as a pool of their own
    ref, rs, mag, smag = ref_linear(q[-280:].cpu(), k[-280:].cpu(), v[-280:].cpu(), decay[-280:].cpu(),
                                    states[-4:].cpu(), torch.tensor([3, -1, 2]), torch.tensor([1, 0, 2]),
                                    starts[1:].cpu() - (t - 280), 0.1)
    n = pa.pa_linear_prefill_workspace_size(4, t, t, hkv, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pa.pa_linear_prefill(out, q, k, v, decay, states, src, dst, starts, 0.1, t, ws)
    assert bool((out[:9] == 7.0).all())
    check_out(out[-280:].cpu(), ref, mag)
    check_states(states[-4:].cpu(), rs, smag, out.dtype)
    # one token of each sequence, of rows a long way apart
    wide = torch.empty(130, 1 << 24, dtype=torch.float16, device="cuda")
    row = 4 * d + 2 * hkv * d
    wide[:, :row] = torch.randn(130, row, generator=g).half().cuda()
    q, k, v = wide[:, :row].split([4 * d, hkv * d, hkv * d], dim=1)
    q, k, v = q.view(130, 4, d), k.view(130, hkv, d), v.view(130, hkv, d)
    src = torch.full((130,), -1, dtype=torch.int32, device="cuda")
    dst, decay = src.clone(), decay[-130:].contiguous()
    src[-2:], dst[-2:] = ns - 2, ns - 2
    src[-2], dst[-2] = ns - 3, ns - 1
    out = torch.full((130, 4, d), 7.0, dtype=torch.float16, device="cuda")
    old = states[-4:].cpu()
    ref, rs, mag, smag = ref_linear(q[-2:].cpu(), k[-2:].cpu(), v[-2:].cpu(), decay[-2:].cpu(), old,
                                    torch.tensor([1, 2]), torch.tensor([3, 2]), torch.tensor([0, 1, 2]), 0.1)
    pa.pa_linear_decode(out, q, k, v, decay, states, src, dst, 0.1)
    assert bool((out[:-2] == 7.0).all())
    check_out(out[-2:].cpu(), ref, mag)
    check_states(states[-4:].cpu(), rs, smag, out.dtype)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (9, 1), (34, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_few_tokens(pa, heads, kv_heads, d, dtype):
    """Speculated tokens, at most 16 a sequence, with more heads a group than one pass
    over the state takes; a padding row and a sequence past its bound among them."""
    x = inputs([16, 3, 0, 9, 1, 2, 15], heads, kv_heads, d, dtype, "token", seed=31, fresh=(3,),
               fused=True, tail=2)
    x["dst"][5] = -1
    check(pa, x, prefill)
    y = inputs([4, 16, 2], heads, kv_heads, d, dtype, "head", seed=32)
    before, out = y["states"].clone(), torch.full_like(y["q"], 7.0)
    prefill(pa, y, out=out, most=15)
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
    assert bool((out[4:20] == 7.0).all()) and not bool((out[:4] == 7.0).all())
    assert torch.equal(y["states"][int(y["dst"][1])], before[int(y["dst"][1])])


@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (6, 2)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_sequences(pa, heads, kv_heads, dtype):
    """More chains than SMs, in the order of lengths (up to 32 sequences) and in their own,
    with padding rows and empty sequences, whose tiles are asked for ahead as well."""
    for b, seed in ((32, 33), (70, 34)):
        lens = [(37 * i * i + 11 * i) % 290 for i in range(b)]
        lens[5] = lens[b - 1] = 0
        x = inputs(lens, heads, kv_heads, 64, dtype, "token", seed=seed, fresh=range(0, b, 4))
        x["dst"][7] = x["dst"][b - 3] = -1
        check(pa, x, prefill)


def test_graphs_share_a_workspace(pa):
    """Two captured calls with cut prompts on one workspace, replayed in turn: the same bits
    as eager calls on a workspace of their own."""
    xs = [inputs(lens, 8, 2, 128, "bf16", "token", seed=35 + i) for i, lens in enumerate(([2500], [900, 1800]))]
    ws = max((workspace(pa, x) for x in xs), key=len)
    assert len(ws) > 256
    outs, wants, graphs = [], [], []
    for x in xs:
        most = longest(x)
        eager = {**x, "states": x["states"].clone()}
        wants.append((prefill(pa, eager), eager["states"]))
        x["before"] = x["states"].clone()
        outs.append(torch.full_like(x["q"], 7.0))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            prefill(pa, x, out=outs[-1], most=most, ws=ws)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            prefill(pa, x, out=outs[-1], most=most, ws=ws)
    for i in (0, 1, 1, 0):
        xs[i]["states"].copy_(xs[i]["before"])
        outs[i].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(outs[i], wants[i][0]) and torch.equal(xs[i]["states"], wants[i][1])
    assert pa.pa_device_errors(clear=True) == 0


def test_host_threads(pa):
    """Four threads, a stream and a workspace each: the bits of one thread alone."""
    def inputs_of(i):
        return (inputs([300 + i, 40], 4, 2, 64, "fp16", "token", seed=40 + i),
                inputs([1] * 5, 4, 2, 64, "fp16", "token", seed=50 + i))

    wants = []
    for i in range(4):
        x, y = inputs_of(i)
        wants.append((prefill(pa, x), x["states"], decode(pa, y), y["states"]))
    work = [inputs_of(i) for i in range(4)]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def run(i):
        try:
            x, y = work[i]
            first = [t["states"].clone() for t in (x, y)]
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                for _ in range(20):
                    for t, s in zip((x, y), first):
                        t["states"].copy_(s)
                    a, b = prefill(pa, x), decode(pa, y)
                stream.synchronize()
            got[i] = (a, x["states"], b, y["states"])
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for g, w in zip(got, wants):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens", [[300], [1200]], ids=str)
def test_channels_of_different_sizes(pa, lens, dtype):
    """Value channels 2^14 apart keep the precision of their own size: a chunk's values and
    a state are scaled as a whole in fp16, and parts of 22 bits reach 2^-39 of the largest,
    2^-25 of the small ones."""
    x = inputs(lens, 4, 2, 128, dtype, "token", seed=60)
    x["v"][..., ::3] *= 2.0 ** -8
    x["v"][..., 1::3] *= 2.0 ** 6
    x["states"][..., ::3] *= 2.0 ** -8
    x["states"][..., 1::3] *= 2.0 ** 6
    check(pa, x, prefill)
