"""The gated delta rule, the query and key norms and the block norms run together, as a model's layers use them (the example
model with mixer="delta"): a training step's gradients against the same model in plain float64 operations, and ragged
prompts continued token by token from pooled states against whole prompts.

The model rounds activations and weights to bfloat16 (2^-8 relative at most, a quarter of that in the mean).  Of these
roundings about 9 a layer lie on a path forwards, as many backwards, and 5 of weights: 41, which add up like independent
errors to 41^0.5 2^-10 = 0.6 % of a gradient's norm.  Norms, gates and the softmax pass an error on with a factor of up to
2 a layer, over 2 layers and the loss: 8 times 0.6 %: 5 % of the norm, for the logits alike.  A missing or wrong term
changes a gradient by tens of per cent.
"""
import os
import sys

import pytest
import torch
import torch.nn.functional as nnf

import delta_reference as ref
import qk_reference

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import linear_attention_lm as lm  # noqa: E402

BAR = 0.05


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plain_logits(p, tokens):
    """The model in plain float64 operations (parameters as given)."""
    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
    x, h = p["embed"][tokens], 0.0
    layers, heads, dim = 2, p["log_decay"].numel(), x.shape[-1]
    for i in range(layers):
        h = h + x
        z = norm(h, p[f"norm.{i}"]) @ p[f"w_in.{i}"]
        q, k, v, gate, raw_g, raw_b = z.split([dim] * 4 + [heads] * 2, -1)
        q, k, v = (a.unflatten(-1, (heads, -1)) for a in (q, k, v))
        q, k = (qk_reference.qk_norm(a, norm="l2", inv_freq=p["inv_freq"]) for a in (q, k))
        o, _ = ref.delta(q, k, v, p["log_decay"] * nnf.softplus(raw_g), torch.sigmoid(raw_b), (dim // heads) ** -0.5)
        w = p[f"head_norm.{i}"].unflatten(-1, (heads, -1))
        x = (norm(o, w).flatten(-2) * nnf.silu(gate)) @ p[f"w_out.{i}"]
    return norm(h + x, p[f"norm.{layers}"]) @ p["unembed"]


def distance(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


def test_training_step_against_plain_operations():
    torch.manual_seed(1)
    model = lm.Model(vocab=64, dim=128, heads=4, mixer="delta")
    tokens = torch.randint(64, (2, 71), device="cuda")
    logits = model(tokens[:, :-1])
    nnf.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten()).backward()
    state = {n: t.detach().double().cpu() for n, t in model.state_dict().items()}
    for n in state:
        state[n].requires_grad_(n not in ("log_decay", "inv_freq"))
    want = plain_logits(state, tokens[:, :-1].cpu())
    nnf.cross_entropy(want.flatten(0, 1), tokens[:, 1:].flatten().cpu()).backward()
    assert distance(logits.detach(), want.detach()) <= BAR
    for n, p in model.named_parameters():
        d = distance(p.grad, state[n].grad)
        print(f"{n}: {d:.3f}", flush=True)
        assert d <= BAR, (n, d)


def test_training_runs():
    torch.manual_seed(0)
    losses, _ = lm.train(lm.Model(mixer="delta"), 4, 4, 100, report=lambda s: None)
    assert all(torch.isfinite(torch.tensor(x)) for x in losses)


def test_steps_from_pooled_states_equal_whole_prompts():
    torch.manual_seed(2)
    model = lm.Model(mixer="delta")
    prompts = torch.randint(model.vocab, (5, 96), device="cuda")
    lengths = torch.tensor([96, 1, 64, 65, 17], device="cuda", dtype=torch.int32)
    tokens, seen = lm.generate(model, prompts, lengths, 12)
    with torch.no_grad():
        for b, n in enumerate(lengths.tolist()):
            whole = torch.cat([prompts[b, :n], tokens[b]])[None]
            want = model(whole)[0, n - 1:-1].double().cpu()
            assert distance(seen[b], want) <= BAR, b


def test_idle_rows_leave_the_pool_alone():
    torch.manual_seed(3)
    model = lm.Model(mixer="delta")
    pool = [torch.randn_like(s) for s in model.new_pool(4)]
    before = [s.clone() for s in pool]
    tokens = torch.randint(model.vocab, (3,), device="cuda")
    at = torch.tensor([7, 0, 100000], device="cuda", dtype=torch.int32)
    logits = model.step(tokens, pool, torch.tensor([2, -1, 0], device="cuda", dtype=torch.int32), at)
    assert torch.isfinite(logits).all()
    for s, s0 in zip(pool, before):
        assert torch.equal(s[[1, 3]], s0[[1, 3]]) and not torch.equal(s[[0, 2]], s0[[0, 2]])
