"""The gated delta rule with a decay of 0 at many tokens of a chunk, as packed short documents have it.

Keys are unit vectors of one token each, so that nothing meets but the token before: q_t = k_{t-1} makes o_t = scale
exp(g_t) v_{t-1}, in which every product but the decay's is exact.  The decay is formed as a hardware power of two
(2^-23), its low part's first-order factor (half of (2^-11 log 2)^2: sums of 32 decays of 0 stay below 2^13, where a
float32 pair's low parts are at most 2^-12 each) and three roundings (the factor, the scale, the product): 2^-23 +
2^-24 + 3 * 2^-24 = 3.6e-7, and g itself times 1 / log 2 is taken in float64.  The bound is 2^-21 = 4.8e-7.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -21


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _inputs(every, L=192):
    gen = torch.Generator().manual_seed(every)
    k = torch.eye(64).repeat(L // 64, 1)[None, :, None]                  # [1, L, 1, 64]
    q = torch.zeros_like(k)
    q[:, 1:] = k[:, :-1]
    v = 1.0 + torch.randint(0, 8, (1, L, 1, 64), generator=gen).float()
    g = -0.3 * torch.rand(1, L, 1, generator=gen) - 0.01
    g[:, ::every] = float("-inf")
    return q, k, v, g, torch.ones(1, L, 1)


@pytest.mark.parametrize("every", [2, 3, 4, 16])
@pytest.mark.parametrize("low", [float("-inf"), -1e5, -130.0])
def test_decays_between_resets(every, low):
    ssm = _ssm()
    q, k, v, g, beta = _inputs(every)
    g = g.clamp(min=low)
    out, _ = ssm.gated_delta_fwd(*(x.cuda() for x in (q, k, v, g, beta)), 0.125)
    want = torch.zeros_like(v, dtype=torch.float64)
    want[:, 1:] = 0.125 * g[:, 1:, :, None].double().exp() * v[:, :-1].double()
    reset = torch.zeros(v.shape[1], dtype=torch.bool)
    reset[::every] = True
    got = out.double().cpu()
    assert not got[:, reset].any()
    e = ((got - want).abs() / want.abs())[:, ~reset]
    print(f"{every}: {float(e.max()):.2e}", flush=True)
    assert float(e.max()) <= BOUND


@pytest.mark.parametrize("every", [2, 3, 4, 16])
def test_gradients_between_resets(every):
    """dv_{t-1} = beta scale exp(g_t) dout_t: one token's output sees one token's value."""
    ssm = _ssm()
    q, k, v, g, beta = _inputs(every)
    got = ssm.gated_delta_bwd(*(x.cuda() for x in (q, k, v, g, beta)), v.cuda(), 0.125)["dv"].double().cpu()
    want = torch.zeros_like(v, dtype=torch.float64)
    want[:, :-1] = 0.125 * g[:, 1:, :, None].double().exp() * v[:, 1:].double()
    seen = torch.ones(v.shape[1], dtype=torch.bool)
    seen[-1] = False
    seen[[t - 1 for t in range(every, v.shape[1], every)]] = False       # what a decay of 0 hides
    assert not got[:, ~seen].any()
    e = ((got - want).abs() / want.abs())[:, seen]
    print(f"{every}: {float(e.max()):.2e}", flush=True)
    assert float(e.max()) <= BOUND
