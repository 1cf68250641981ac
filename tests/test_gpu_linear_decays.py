"""Decays of linear attention over their whole range, against the 64-bit recurrence."""
import math

import pytest
import torch

from tests._linear_ref import check_out, check_states, inputs, ref_linear
from tests.test_gpu_linear import decode, pa, prefill  # noqa: F401

pytestmark = pytest.mark.gpu

RATES = [-0.5, -0.69, -0.6931471, -0.6931472, -0.6931473, -0.7, -1.0, -2.0, -4.0, -6.0, -8.0, -10.0,
         -12.0, -14.0, -16.0, -17.0, -17.5, -18.0, -20.0, -25.0, -30.0, -80.0]


@pytest.mark.parametrize("run,lens", [(decode, [1] * 3), (prefill, [1, 2, 5, 16])], ids=["step", "few"])
@pytest.mark.parametrize("new", [True, False], ids=["new", "decay alone"])
@pytest.mark.parametrize("d", [64, 128])
def test_strong_decays(pa, run, lens, new, d):
    """A decayed state is right relative to what is left of it, with k v^T or without.

    A step token by token: e^g is off by 2^-23 of itself (exp, and e^g - 1 where e^g is at
    least a half), its product with the state and the sum by 2^-24 each: 2^-22 of the sum
    of absolute values a step.  Numbers below 2^-126 have steps of 2^-149."""
    n = len(RATES)
    x = inputs(lens, n, n, d, "fp16", "head", seed=80)
    x["log_decay"] = torch.tensor(RATES, device="cuda")
    if not new:
        x["v"].zero_()
    ref, states, mag, smag = ref_linear(*(x[k] for k in ("q", "k", "v", "log_decay", "states", "src",
                                                         "dst", "starts", "scale")))
    out = run(pa, x)
    to = x["dst"].long()
    err = (x["states"].double() - states).abs()[to]
    steps = torch.tensor(lens, device="cuda")[:, None, None, None]
    tol = steps * (2.0 ** -22 * smag[to] + 2.0 ** -148)
    assert not (err > tol).any(), [(r, float((err / tol)[:, i].max())) for i, r in enumerate(RATES)]
    check_out(out, ref, mag)
    assert pa.pa_device_errors(clear=True) == 0
    assert math.isfinite(float(out.float().sum()))


@pytest.mark.parametrize("every", [2, 3, 4, 8])
@pytest.mark.parametrize("strong", [-20.0, -1e4, -math.inf])
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_ordinary_tokens_between_strong_decays(pa, every, strong, heads, dtype):
    """The weight of a token for one that follows is that of the decays between them,
    however strong the ones before.

    All scores are equal and values are 1 or -1, so that many outputs are small differences
    of terms that are not, and only those terms' errors show.  The tolerance is that of
    tests/_linear_ref.py; its exponents' part, for sums of up to 31 terms that are off by
    2^-24 of the sum x each, with |x| e^-|x| <= 0.37, is 31 * 0.37 * 2^-24 < 2^-20, and the
    other parts are below 2^-19 + 2^-21."""
    d = 64
    x = inputs([300, 129, 40], 2 * heads, 2, d, dtype, "token", seed=81, fresh=(0,))
    g = x["log_decay"]
    g.uniform_(-0.02, 0.0, generator=torch.Generator("cuda").manual_seed(every))
    g[every // 2::every, 0] = strong
    g[torch.rand(len(g), generator=torch.Generator().manual_seed(every)).cuda() < 1 / every, 1] = strong
    x["q"].fill_(1.0)
    x["k"].fill_(1.0)
    x["v"].copy_(x["v"].sign())
    x["states"].sign_()
    ref, states, mag, smag = ref_linear(*(x[k] for k in ("q", "k", "v", "log_decay", "states", "src",
                                                         "dst", "starts", "scale")))
    out = prefill(pa, x)
    check_out(out, ref, mag)
    check_states(x["states"], states, smag, out.dtype)
    assert pa.pa_device_errors(clear=True) == 0
