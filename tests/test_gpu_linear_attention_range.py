"""Linear attention at the ends of float32's range, and with decays on both sides of 1: results are finite and
right wherever the recurrence is, so no scaling on the way may overflow or vanish.

Errors, rows and bounds are those of the parity tests: 5e-5 in float32 and of states, 1.6e-2 of bfloat16 outputs."""
import pytest
import torch

import lm_reference as ref
from test_gpu_linear_attention import STATE, _check, _cuda, _inputs, _ssm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _both(t, g, s0, df, scale, dtype, unit_of):
    """The prompt form and its gradient against the recurrence; the size of every result is divided out first."""
    ssm = _ssm()
    d = _cuda(t)
    s0c, dfc = (None if x is None else x.cuda() for x in (s0, df))
    out, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), scale, initial_state=s0c)
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, scale, s0)
    got = dict(out=out, final_state=fin)
    got.update(ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], scale, initial_state=s0c,
                                        dfinal_state=dfc, want_dinitial_state=True))
    want = dict(out=want, final_state=wfin, **ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], scale, s0, df))
    for n in want:
        unit = unit_of[n]
        assert float(want[n].abs().max()) < 1e38            # (the case stays in range itself)
        _check(got[n].double() / unit, want[n] / unit, dtype, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e35, 1e30, 1e-28])
@pytest.mark.parametrize("L,K,V", [(700, 64, 64), (1300, 64, 64), (330, 128, 128), (130, 40, 24)])
def test_values_at_the_ends_of_the_range(L, K, V, size, dtype):
    # memories of 32 tokens and of 4096; v and the output gradient carry the size.  (The decayed values of
    # bfloat16 rows are split: three terms of 1e-28 still have their bits.)  Two heads, so that the longer
    # ones run in segments
    t, _, s0, df = _inputs(1, L, 2, K, V, dtype, seed=L + K)
    g = torch.log1p(-torch.tensor([1.0 / 32, 1.0 / 4096]))
    t["v"], t["do"] = ((t[n].float() * size).to(dtype) for n in ("v", "do"))
    s0, df = s0 * size, df * size
    # dq = S do and dk = G v are products of two such values: one of them is left at 1 in turn
    one = dict(t, v=(t["v"].float() / size).to(dtype))
    two = dict(t, do=(t["do"].float() / size).to(dtype))
    units = dict(out=1, final_state=1, dq=size, dk=size, dv=size, dinitial_state=size)
    _both(one, g, s0 / size, df, 1.0 / 8, dtype, units)
    units = dict(out=size, final_state=size, dq=size, dk=size, dv=1, dinitial_state=1)
    _both(two, g, s0, df / size, 1.0 / 8, dtype, units)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("log_decay", [1e-3, 0.05, 0.4])
@pytest.mark.parametrize("L", [200, 1100])
def test_states_that_grow(L, log_decay, dtype):
    # lam > 1: the last tokens' outputs are the largest, by far, and each row is measured by its own size
    if log_decay * L > 60:
        L = int(60 / log_decay)                             # (e^60 = 1e26)
    t, _, s0, df = _inputs(1, L, 2, 64, 64, dtype, seed=L)
    g = torch.tensor([log_decay, log_decay / 2])
    d = _cuda(t)
    out, fin = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda())
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, 0.125, s0)
    size = want.norm(dim=-1, keepdim=True)
    _check(out.double().cpu() / size, want / size, dtype, "out")
    _check(fin, wfin, dtype, "final_state")
    got = _ssm().linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                      dfinal_state=df.cuda())
    for n, w in ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], 0.125, s0, df).items():
        size = w.norm(dim=-1, keepdim=True)
        _check(got[n].double().cpu() / size, w / size, dtype, n)


def test_infinite_states_stay_infinite():
    # float32: an infinite entry of the state is scaled by lam^64 again and again and stays infinite, not a NaN
    H, K, V, L = 2, 64, 64, 600
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, L, H, K, generator=gen) for _ in range(3))
    g = torch.log1p(-torch.tensor([1.0 / 32, 1.0 / 4096]))
    s0 = torch.randn(1, H, K, V, generator=gen)
    s0[:, :, 3, 5], s0[:, :, 60, 63] = float("inf"), float("-inf")
    for n in (64, 130, L):
        for heads in (H, 1):                                # (one segment, then several)
            _, fin = _ssm().linear_attention_fwd(q[:, :n, :heads].cuda(), k[:, :n, :heads].cuda(), v[:, :n, :heads].cuda(),
                                                 g[:heads].cuda(), initial_state=s0[:, :heads].contiguous().cuda())
            fin = fin.cpu()
            assert torch.equal(torch.isinf(fin), torch.isinf(s0[:, :heads])) and not torch.isnan(fin).any()
            assert torch.equal(fin.sign()[torch.isinf(fin)], s0[:, :heads].sign()[torch.isinf(fin)])
            _, want = ref.attention(q[:, :n, :heads], k[:, :n, :heads], v[:, :n, :heads], g[:heads], 1.0, s0[:, :heads])
            fine = torch.isfinite(want)
            assert float((fin.double() - want)[fine].norm() / want[fine].norm()) <= STATE


def test_no_token_leaves_the_smallest_states_alone():
    # scaling is for rows with tokens: a state below what scaled registers hold comes back as it was
    s0 = torch.full((2, 1, 64, 64), 3e-38)
    s0[..., 1::2] = 1e-40
    x = torch.randn(2, 70, 1, 64).cuda()
    _, fin = _ssm().linear_attention_fwd(x, x, x, torch.tensor([-0.5]).cuda(), initial_state=s0.cuda(),
                                         lengths=torch.tensor([70, 0], dtype=torch.int32).cuda())
    assert torch.equal(fin[1].cpu(), s0[1])
