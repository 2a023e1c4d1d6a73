"""How a call is put together does not show in its results: the same bits from rows of any alignment and
strides, and with or without the states asked for, in one segment and in several."""
import pytest
import torch

from test_gpu_linear_attention import _inputs, _ssm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _at(t, offset):
    """A copy of t whose rows start `offset` elements past a 16-byte boundary, and lie as far apart."""
    wide = torch.empty(*t.shape[:-2], t.shape[-2] * t.shape[-1] + 8 + offset, dtype=t.dtype, device="cuda")
    view = wide[..., offset:offset + t.shape[-2] * t.shape[-1]].unflatten(-1, t.shape[-2:])
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,H,K,V", [(330, 2, 64, 64), (1300, 2, 64, 64), (1300, 3, 128, 128), (300, 2, 96, 128),
                                     (1100, 2, 128, 64)])
def test_same_bits(L, H, K, V, dtype):
    ssm = _ssm()
    t, g, s0, df = _inputs(1, L, H, K, V, dtype, seed=L)
    g, s0, df = g.cuda(), s0.cuda(), df.cuda()
    segmented = ssm.linear_attention_workspace_size(1, L, H, K, V, dtype) > 0
    assert segmented == (L > 1000)
    d = {n: x.cuda() for n, x in t.items()}
    out, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g, initial_state=s0)
    alone, none = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g, initial_state=s0, return_final_state=False)
    assert none is None and torch.equal(alone, out)
    grads = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g, d["do"], initial_state=s0, dfinal_state=df)
    alone = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g, d["do"], initial_state=s0, dfinal_state=df,
                                     want_dinitial_state=False)
    assert alone["dinitial_state"] is None
    assert all(torch.equal(grads[n], alone[n]) for n in ("dq", "dk", "dv"))
    for offset in (1, 2):
        v = {n: _at(x, offset) for n, x in t.items()}
        o, f = ssm.linear_attention_fwd(v["q"], v["k"], v["v"], g, initial_state=s0)
        assert torch.equal(o, out) and torch.equal(f, fin), offset
        got = ssm.linear_attention_bwd(v["q"], v["k"], v["v"], g, v["do"], initial_state=s0, dfinal_state=df)
        assert all(torch.equal(got[n], grads[n]) for n in grads), offset
