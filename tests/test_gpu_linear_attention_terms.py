"""The bits that bfloat16 calls carry on the way, which an output's own rounding would hide, and the widest tiles
over many chunks.

Scores and states as operands of the output are two bfloat16 terms: sums of 1 + 2^-12 and -1 give 2^-12 exactly, where
one term would give 0.  The decayed values that enter a returned state are three: a state lam^n is held to the error
of its weight, of which there are at most three hardware exponentials (2 units of 2^-24 each), six products and
their arguments' rounding (n log2(lam) below 2: 3 units), under 16 units; twice that, 2e-6, is the bar.  Two terms
leave up to 2^-17 = 7.6e-6, and among 64 heads some come near it."""
import pytest
import torch

import test_gpu_linear_attention as base
from test_gpu_linear_attention import _check, _cuda, _inputs, _ssm
import lm_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TINY = 2.0 ** -12


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rows(L, width, at):
    """[1, L, 1, width] bfloat16 zeros with rows of values at tokens."""
    t = torch.zeros(1, L, 1, width)
    for token, values in at.items():
        t[0, token, 0, :len(values)] = torch.tensor(values)
    return t.to(BF16).cuda()


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("first,second,L", [(0, 1, 64), (3, 40, 64), (33, 62, 70), (70, 100, 130)])
def test_scores_keep_16_bits(first, second, L, width):
    # (1 + 2^-12) of one token and -1 of another, in the output and in each gradient
    ssm = _ssm()
    decay = torch.zeros(1, device="cuda")
    fine, plain = [1.0, 2.0 ** -6], [1.0]
    plus, minus = [1.0] * width, [-1.0] * width
    every = _rows(L, width, {t: fine for t in range(L)})
    scores, values = _rows(L, width, {first: fine, second: plain}), _rows(L, width, {first: plus, second: minus})
    out, _ = ssm.linear_attention_fwd(every, scores, values, decay, 1.0)
    assert torch.equal(out[0, second:].float(), torch.full((L - second, 1, width), TINY, device="cuda"))
    # dq_i = sum (dout_i . v_j) k_j;  dk_j = sum (v_j . dout_i) q_i and dv_j = sum (k_j . q_i) dout_i over later i
    got = ssm.linear_attention_bwd(every, values, scores, decay, every, 1.0)
    assert torch.equal(got["dq"][0, second:].float(), torch.full((L - second, 1, width), TINY, device="cuda"))
    back = {first: plain, second: fine}
    scores, values = _rows(L, width, back), _rows(L, width, {first: minus, second: plus})
    got = ssm.linear_attention_bwd(values, every, every, decay, scores, 1.0)
    assert torch.equal(got["dk"][0, :first + 1].float(), torch.full((first + 1, 1, width), TINY, device="cuda"))
    got = ssm.linear_attention_bwd(scores, every, every, decay, values, 1.0)
    assert torch.equal(got["dv"][0, :first + 1].float(), torch.full((first + 1, 1, width), TINY, device="cuda"))


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("L", [5, 64, 200, 1100])
def test_states_as_operands_keep_16_bits(L, width):
    # a state with rows of 1 + 2^-12 and -1, carried over L tokens that add nothing
    ssm = _ssm()
    decay, zero = torch.zeros(1, device="cuda"), _rows(L, width, {})
    both = _rows(L, width, {t: [1.0, 1.0] for t in range(L)})
    s0 = torch.zeros(1, 1, width, width, device="cuda")
    s0[0, 0, 0], s0[0, 0, 1] = 1.0 + TINY, -1.0
    want = torch.full((1, L, 1, width), TINY, device="cuda")
    out, fin = ssm.linear_attention_fwd(both, zero, zero, decay, 1.0, initial_state=s0)
    assert torch.equal(out.float(), want) and torch.equal(fin, s0)
    across = s0.transpose(2, 3).contiguous()
    got = ssm.linear_attention_bwd(zero, zero, zero, decay, both, 1.0, initial_state=across)
    assert torch.equal(got["dq"].float(), want)
    got = ssm.linear_attention_bwd(zero, zero, both, decay, zero, 1.0, dfinal_state=across)
    assert torch.equal(got["dk"].float(), want)
    got = ssm.linear_attention_bwd(zero, both, zero, decay, zero, 1.0, dfinal_state=s0)
    assert torch.equal(got["dv"].float(), want)


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("L,token", [(21, 0), (64, 10), (70, 5), (600, 550), (1100, 1060)])
def test_states_that_are_returned_keep_24_bits(L, token, width):
    ssm = _ssm()
    H = 64 if L < 1000 else 2                               # (two heads of 1100 tokens run in segments)
    n = L - 1 - token
    worst = 0.0
    for part in range(64 // H):
        power = torch.linspace(0.5, 1.3, 64, dtype=torch.float64)[part * H:(part + 1) * H] / n
        decay = (-power).float().cuda()
        x = torch.zeros(1, L, H, width, dtype=BF16, device="cuda")
        x[0, token] = 1.0
        zero = torch.zeros_like(x)
        _, fin = ssm.linear_attention_fwd(zero, x, x, decay, 1.0)
        want = torch.exp(decay.double() * n).view(1, H, 1, 1)
        worst = max(worst, float(((fin.double() - want) / want).abs().max()))
        # backwards the state decays once more, past the token
        y = x.flip(1)
        got = ssm.linear_attention_bwd(y, zero, zero, decay, y, 1.0, want_dinitial_state=True)["dinitial_state"]
        want = torch.exp(decay.double() * (n + 1)).view(1, H, 1, 1)
        worst = max(worst, float(((got.double() - want) / want).abs().max()))
    print(f"L {L} width {width}: {worst:.2e}", flush=True)
    assert worst <= 2e-6


# ---- tiles of 128 x 128 with every column there, over several whole chunks, in one segment and in several

WIDE = [(1, 330, 2, 128, 128, None), (2, 257, 4, 128, 128, (2, 1, 4)), (1, 1300, 2, 128, 128, None),
        (1, 1408, 3, 128, 128, (3, 1, 1)), (1, 450, 2, 64, 64, None), (1, 400, 2, 128, 64, None), (1, 400, 2, 64, 128, None)]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("shape", WIDE)
def test_forward_over_many_chunks(shape, dtype):
    base.test_forward(*shape, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("shape", WIDE)
def test_gradient_over_many_chunks(shape, dtype):
    base.test_gradient(*shape, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("L,lengths", [(330, (330, 0, 193, 256)), (1300, (1300, 1, 700, 1279))])
def test_ragged_over_many_chunks(L, lengths, dtype):
    ssm = _ssm()
    t, g, s0, df = _inputs(4, L, 2, 128, 128, dtype, seed=L)
    absent = torch.arange(L)[None] >= torch.tensor(lengths)[:, None]
    for x in t.values():
        x[absent] = float("nan")
    d, n = _cuda(t), torch.tensor(lengths, dtype=torch.int32).cuda()
    got = dict(zip(("out", "final_state"), ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda(),
                                                                    lengths=n)))
    got.update(ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                        dfinal_state=df.cuda(), lengths=n))
    want = dict(zip(("out", "final_state"), ref.attention(t["q"], t["k"], t["v"], g, 128 ** -0.5, s0, lengths)))
    want.update(ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], 128 ** -0.5, s0, df, lengths))
    for name in want:
        _check(got[name], want[name], dtype, name)
