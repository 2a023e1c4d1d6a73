"""A value that is not finite reaches what the recurrence says and nothing else: outputs (and gradients, walked
backwards) before its token are those of the other values, in its own chunk of tokens too.

Finite results are held to the parity tests' bounds; where the recurrence is not finite, neither is the result."""
import pytest
import torch

import lm_reference as ref
from test_gpu_linear_attention import OUT, STATE, _check, _cuda, _inputs, _ssm

pytestmark = pytest.mark.gpu

BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf")}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _same(got, want, dtype, name):
    """The parity tests' error with the rows that are not finite left out of a head's mean size as well."""
    fine = torch.isfinite(want)
    got = got.cpu()
    assert torch.equal(torch.isfinite(got), fine), name
    keep = lambda t: torch.where(fine, t.double(), 0.0)
    error, size, rows = (keep(got) - keep(want)).norm(dim=-1), keep(want).norm(dim=-1), fine.any(-1)
    axes = (0, 1) if rows.dim() == 3 else (0, 2)
    mean = (size.square().sum(axes, keepdim=True) / rows.sum(axes, keepdim=True).clamp(min=1)).sqrt()
    worst = float((error / mean.clamp(min=1e-30)).max())
    print(f"{name} {tuple(got.shape)} {dtype}: {worst:.2e}, {int(fine.sum())} finite", flush=True)
    assert worst <= (STATE if "state" in name else OUT[dtype]), (name, worst)
    return int(fine.sum())


def _both(t, g, s0, df, dtype, lengths=None):
    ssm = _ssm()
    d = _cuda(t)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    got = dict(zip(("out", "final_state"), ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), 0.125,
                                                                    initial_state=s0.cuda(), lengths=n)))
    got.update(ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], 0.125, initial_state=s0.cuda(),
                                        dfinal_state=df.cuda(), lengths=n))
    want = dict(zip(("out", "final_state"), ref.attention(t["q"], t["k"], t["v"], g, 0.125, s0, lengths)))
    want.update(ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], 0.125, s0, df, lengths))
    return {n: _same(got[n], want[n], dtype, n) for n in want}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
@pytest.mark.parametrize("token,value", [(0, "nan"), (1, "inf"), (31, "nan"), (32, "-inf"), (63, "nan"), (64, "inf"),
                                         (100, "nan"), (149, "inf")])
def test_one_value(token, value, name, dtype):
    t, g, s0, df = _inputs(2, 150, 2, 64, 64, dtype, seed=token)
    t[name][1, token, 0, 37] = BAD[value]
    _both(t, g, s0, df, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,H,K,V,heads", [(330, 2, 128, 128, None), (1300, 2, 128, 128, None), (1100, 1, 64, 64, None),
                                           (200, 4, 64, 128, (4, 2, 2)), (130, 6, 128, 64, (2, 6, 3)), (129, 2, 33, 17, None),
                                           (1050, 1, 100, 36, None), (77, 3, 72, 40, (1, 1, 3))])
@pytest.mark.parametrize("name", ["k", "v", "do"])
def test_shapes(L, H, K, V, heads, name, dtype):
    # two tokens of one chunk in different columns, of which the second comes late in the sequence
    t, g, s0, df = _inputs(1, L, H, K, V, dtype, heads, seed=L + V)
    width, last = t[name].shape[-1], t[name].shape[-2] - 1
    t[name][0, L // 2, 0, 0] = BAD["nan"]
    t[name][0, L // 2 + 3, last, width - 1] = BAD["inf"]
    t[name][0, L - 2, last, width // 2] = BAD["nan"]
    counts = _both(t, g, s0, df, dtype)
    if name == "v":
        assert counts["out"] > (L // 2) * H * V             # everything before is there, and other columns after it


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_absent_tokens_beside_them(dtype):
    t, g, s0, df = _inputs(3, 150, 2, 64, 72, dtype, seed=5)
    lengths = [150, 90, 64]
    for n in "kv":
        t[n][0, 149, 1, 3], t[n][1, 70, 0, 8], t[n][2, 63, 0, 0] = BAD["nan"], BAD["inf"], BAD["nan"]
        t[n][1, 95:], t[n][2, 64:] = BAD["nan"], BAD["-inf"]                   # (absent)
    _both(t, g, s0, df, dtype, lengths)


def test_whole_rows_and_the_smallest_value():
    # every value of a token, and a token of the type's lowest (finite) value, whose products overflow
    t, g, s0, df = _inputs(1, 100, 2, 64, 64, torch.float32, seed=6)
    t["v"][0, 50] = BAD["nan"]
    _both(t, g, s0, df, torch.float32)
    out, _ = _ssm().linear_attention_fwd(*(x.cuda() for x in (t["q"], t["k"])),
                                         torch.where(torch.isnan(t["v"]), torch.finfo(torch.float32).min, t["v"]).cuda(),
                                         g.cuda(), 0.125, initial_state=s0.cuda())
    want, _ = ref.attention(t["q"], t["k"], t["v"], g, 0.125, s0)
    _check(out[:, :50], want[:, :50], torch.float32, "out")


def test_the_results_in_place_of_the_state():
    # the state is read again when a head's tokens are walked again
    t, g, s0, _ = _inputs(1, 200, 2, 64, 64, torch.float32, seed=7)
    t["v"][0, 150, 0, 9] = BAD["nan"]
    d, state = _cuda(t), s0.cuda()
    out, fin = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), 0.125, initial_state=state, final_state=state)
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, 0.125, s0)
    _same(out, want, torch.float32, "out")
    _same(fin, wfin, torch.float32, "final_state")
