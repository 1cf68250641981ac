"""Prompts of pa_linear_prefill that are cut into segments: in place, and where the
states that the segments start from come from."""
import pytest
import torch

from tests._linear_ref import check_out, check_states, inputs, ref_linear
from tests.test_gpu_linear import check, pa, prefill, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def lines(x, ws):
    """The workspace as states, one for each segment (and what lies behind them)."""
    shape = x["states"].shape[1:]
    n = len(ws) // (4 * shape.numel())
    return ws[:n * 4 * shape.numel()].view(torch.float32).view(n, *shape)


@pytest.mark.parametrize("lens", [[2100], [300, 5, 1500]], ids=str)
@pytest.mark.parametrize("heads,kv_heads,d", [(2, 2, 64), (8, 2, 128)])
def test_the_last_pass_starts_from_a_copy(pa, lens, heads, kv_heads, d):
    """The CTAs of a pass run in any order, so the pass that writes a cut sequence's state
    must not read it: the state that its first segment starts from is a copy in the
    workspace, of zeros where there is none."""
    for fresh in ((), (0,)):
        x = inputs(lens, heads, kv_heads, d, "bf16", "token", seed=70, fresh=fresh)
        ws = workspace(pa, x)
        ws.fill_(0xAB)
        first = x["states"][int(x["src"][0])].clone() if not fresh else torch.zeros_like(x["states"][0])
        check(pa, x, lambda pa, x: prefill(pa, x, ws=ws))
        copies = (lines(x, ws) == first).flatten(1).all(1)
        assert int(copies.sum()) == 1


@pytest.mark.parametrize("lens,heads,kv_heads,d", [
    ([129, 1, 0, 260], 8, 2, 128),         # last segments of one and of four tokens
    ([3000], 6, 2, 128),
    ([513, 0, 1500, 1, 2049, 40], 6, 2, 64),
    ([5000, 4000], 32, 32, 64),            # more segments than SMs
    ([8200, 500], 16, 16, 128)], ids=str)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_in_place(pa, lens, heads, kv_heads, d, dtype):
    """src_states and dst_states the same: a prompt that goes on."""
    for seed in (71, 72):
        x = inputs(lens, heads, kv_heads, d, dtype, "token", seed=seed)
        x["dst"] = x["src"].clone()
        apart = {**x, "states": x["states"].clone()}
        apart["dst"] = torch.tensor([i for i in range(len(x["states"])) if i not in x["src"].tolist()],
                                    dtype=torch.int32, device="cuda")[:len(lens)]
        out = check(pa, x, prefill)
        assert torch.equal(prefill(pa, apart), out)
        for a, b in zip(x["dst"].tolist(), apart["dst"].tolist()):
            assert torch.equal(x["states"][a], apart["states"][b])


@pytest.mark.parametrize("b,at", [(33, 0), (40, 32), (40, 39), (64, 31), (65, 33), (65, 64), (200, 0),
                                  (200, 97), (200, 199)])
@pytest.mark.parametrize("heads,kv_heads,d,dtype", [(6, 2, 64, "fp16"), (2, 1, 128, "bf16")])
def test_a_long_prompt_among_many(pa, b, at, heads, kv_heads, d, dtype):
    """More sequences than a warp looks through at once, one of them (or two) cut: empty
    ones, padding rows and one past its bound stand before and behind it."""
    lens = [(37 * i * i + 11 * i) % 120 for i in range(b)]
    lens[at] = 4100
    lens[(at + 35) % b] = 700              # segments of its own
    bad = (at + 34) % b
    lens[bad] = 4101                       # longer than max_query_len
    lens[(at + 3) % b] = lens[(at + 33) % b] = 0
    x = inputs(lens, heads, kv_heads, d, dtype, "token", seed=b + at, fresh=range(0, b, 5), tail=3)
    x["dst"][(at + 7) % b] = x["dst"][(at + 40) % b if b > 40 else (at + 9) % b] = -1
    assert at not in (bad, (at + 7) % b)
    ws = workspace(pa, x, 4100)
    ws.fill_(0xAB)
    before = x["states"].clone()
    dst = x["dst"].clone()
    dst[bad] = -1                          # as a padding row: nothing read or written
    ref, states, mag, smag = ref_linear(*(x[k] for k in ("q", "k", "v", "log_decay", "states", "src")),
                                        dst, x["starts"], x["scale"])
    out = prefill(pa, x, most=4100, ws=ws)
    assert bool((ws != 0xAB).any()), "not cut"
    check_out(out, ref, mag)
    check_states(x["states"], states, smag, out.dtype)
    assert bool((out[torch.isnan(mag)] == 7.0).all())
    wrote = dst[dst >= 0].long()
    keep = torch.ones(len(before), dtype=torch.bool, device="cuda")
    keep[wrote] = False
    assert torch.equal(x["states"][keep], before[keep])
    assert pa.pa_device_errors(clear=True) == pa.DEVERR_SEQ_LEN
