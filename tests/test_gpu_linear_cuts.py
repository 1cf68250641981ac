"""Prompts of pa_linear_prefill that are cut into segments: in place, and where the
states that the segments start from come from."""
import pytest
import torch

from tests._linear_ref import inputs
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
