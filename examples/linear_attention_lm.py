"""A small language model of linear attention blocks, trained and then served, on one GPU.

    python examples/linear_attention_lm.py [--steps 80] [--batch 16] [--length 256] [--serve 8]

Every block is

    q, k, v, gate = y W_in;   o = linear attention of q, k, v;   t = norm per head(o) * silu(gate)
    h = h + t W_out;          y = norm(h)   (the norm in front of the next block)

where the attention, both norms, the gate and the residual sum run as the library's kernels, forward and backward, and the
projections are matrix products.  Training shows one step of each; serving runs prompts of unequal lengths at once, keeps
every sequence's states in a pool, and continues them token by token from the pool's slots.  The data are synthetic: a
random permutation of the vocabulary is followed with probability 0.9, else a token is drawn at random.
"""
import argparse
import math
import os
import sys
import time

import torch
import torch.nn.functional as nnf

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_68_amd as ssm  # noqa: E402


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        ctx.save_for_backward(q, k, v, log_decay)
        return ssm.linear_attention_fwd(q, k, v, log_decay, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, dout):
        q, k, v, log_decay = ctx.saved_tensors
        g = ssm.linear_attention_bwd(q, k, v, log_decay, dout)
        return g["dq"], g["dk"], g["dv"], None


class GatedHeadNorm(torch.autograd.Function):
    """norm over each of `heads` column groups of x, times weight, times silu(gate)."""
    @staticmethod
    def forward(ctx, x, gate, weight, heads):
        ctx.save_for_backward(x, gate, weight)
        ctx.heads = heads
        return ssm.block_norm_fwd(x, gate=gate, post_weight=weight, groups=heads)[0]

    @staticmethod
    def backward(ctx, dt):
        x, gate, weight = ctx.saved_tensors
        g = ssm.block_norm_bwd(x, dh=dt.contiguous(), gate=gate, post_weight=weight, groups=ctx.heads)
        return g["dx"], g["dgate"], g["dpost_weight"], None


class AddNorm(torch.autograd.Function):
    """h = residual + x; y = norm(h) * weight."""
    @staticmethod
    def forward(ctx, x, residual, weight):
        h, y = ssm.block_norm_fwd(x, residual, pre_weight=weight)
        ctx.save_for_backward(x, h, weight)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        x, h, weight = ctx.saved_tensors
        g = ssm.block_norm_bwd(x, h, dy.contiguous(), dh.contiguous(), pre_weight=weight, residual_dtype=h.dtype)
        return g["dx"], g["dresidual"], g["dpre_weight"]


class Model(torch.nn.Module):
    def __init__(self, vocab=256, dim=256, heads=4, layers=2, device="cuda"):
        super().__init__()
        self.vocab, self.dim, self.heads, self.layers = vocab, dim, heads, layers
        par = lambda *s, std: torch.nn.Parameter(torch.randn(*s, device=device) * std)
        one = lambda: torch.nn.Parameter(torch.ones(dim, device=device))
        self.embed = par(vocab, dim, std=1.0)
        self.w_in = torch.nn.ParameterList([par(dim, 4 * dim, std=dim ** -0.5) for _ in range(layers)])
        self.w_out = torch.nn.ParameterList([par(dim, dim, std=(2 * layers * dim) ** -0.5) for _ in range(layers)])
        self.head_norm = torch.nn.ParameterList([one() for _ in range(layers)])
        self.norm = torch.nn.ParameterList([one() for _ in range(layers + 1)])
        self.unembed = par(dim, vocab, std=dim ** -0.5)
        # the heads forget at rates from 2^-2 to 2^-2-heads
        rates = torch.log1p(-(2.0 ** -(2.0 + torch.arange(heads, dtype=torch.float32))))
        self.register_buffer("log_decay", rates.to(device))

    def project(self, y, layer):
        """q, k, v [..., heads, dim / heads] and gate [..., dim]: views of one product."""
        z = (y @ self.w_in[layer].to(y.dtype)).unflatten(-1, (4, self.dim))
        q, k, v = (z[..., i, :].unflatten(-1, (self.heads, -1)) for i in range(3))
        return q, k, v, z[..., 3, :]

    def logits(self, y):
        return (y @ self.unembed.to(y.dtype)).float()

    def forward(self, tokens):
        """Training: logits [batch, length, vocab], every kernel inside autograd."""
        x = self.embed[tokens].bfloat16()
        h = torch.zeros(x.shape, device=x.device)
        for i in range(self.layers):
            h, y = AddNorm.apply(x, h, self.norm[i])
            q, k, v, gate = self.project(y, i)
            o = LinearAttention.apply(q, k, v, self.log_decay)
            x = GatedHeadNorm.apply(o.flatten(-2), gate, self.head_norm[i], self.heads) @ self.w_out[i].to(x.dtype)
        h, y = AddNorm.apply(x, h, self.norm[-1])
        return self.logits(y)

    def new_pool(self, slots):
        """One state per layer, slot and head."""
        d = self.dim // self.heads
        return [torch.zeros(slots, self.heads, d, d, device=self.log_decay.device) for _ in range(self.layers)]

    def serve(self, tokens, mix):
        """Logits for tokens [..., length or none]; mix(layer, q, k, v) is the attention of a prompt or of a token."""
        x = self.embed[tokens].bfloat16()
        h = torch.zeros(x.shape, device=x.device)
        y = torch.empty_like(x)
        for i in range(self.layers):
            ssm.block_norm_fwd(x, h, pre_weight=self.norm[i], h=h, y=y)           # h in place
            q, k, v, gate = self.project(y, i)
            o = mix(i, q, k, v).flatten(-2)
            t = ssm.block_norm_fwd(o, gate=gate, post_weight=self.head_norm[i], groups=self.heads)[0]
            x = t @ self.w_out[i].to(x.dtype)
        ssm.block_norm_fwd(x, h, pre_weight=self.norm[-1], h=h, y=y)
        return self.logits(y)

    @torch.no_grad()
    def prefill(self, tokens, lengths, pool, slots):
        """Prompts [batch, length] of `lengths` tokens each; their states go to the pool's `slots`."""
        def mix(i, q, k, v):
            o, state = ssm.linear_attention_fwd(q, k, v, self.log_decay, lengths=lengths)
            pool[i][slots.long()] = state
            return o
        return self.serve(tokens, mix)

    @torch.no_grad()
    def step(self, tokens, pool, slots):
        """One token for every row; a row whose slot is -1 is idle."""
        return self.serve(tokens, lambda i, q, k, v: ssm.linear_attention_step(pool[i], q, k, v, self.log_decay,
                                                                               slots=slots))


def batch_of(permutation, batch, length, generator):
    """[batch, length + 1] tokens: the permutation is followed with probability 0.9."""
    vocab, device = permutation.numel(), permutation.device
    t = torch.randint(vocab, (batch, length + 1), device=device, generator=generator)
    keep = torch.rand(batch, length + 1, device=device, generator=generator) < 0.9
    for i in range(1, length + 1):
        t[:, i] = torch.where(keep[:, i], permutation[t[:, i - 1]], t[:, i])
    return t


def train(model, steps, batch, length, seed=0, report=print):
    """Returns the loss of every step."""
    device = model.log_decay.device
    gen = torch.Generator(device).manual_seed(seed)
    permutation = torch.randperm(model.vocab, device=device, generator=gen)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for i in range(steps):
        t = batch_of(permutation, batch, length, gen)
        loss = nnf.cross_entropy(model(t[:, :-1]).flatten(0, 1), t[:, 1:].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if i % 20 == 0 or i == steps - 1:
            report(f"step {i:4d}: loss {losses[-1]:.3f}")
    return losses, permutation


def generate(model, prompts, lengths, new_tokens):
    """Greedy continuation of prompts [batch, length] (`lengths` tokens each used).  Returns the tokens
    [batch, new_tokens] and the logits each was chosen from [batch, new_tokens, vocab]."""
    batch = prompts.shape[0]
    slots = torch.randperm(2 * batch, device=prompts.device)[:batch].int()        # any free slots of a larger pool
    pool = model.new_pool(2 * batch)
    logits = model.prefill(prompts, lengths.int(), pool, slots)
    last = logits[torch.arange(batch, device=prompts.device), lengths.long() - 1]
    out, seen = [], []
    for _ in range(new_tokens):
        out.append(last.argmax(-1))
        seen.append(last)
        last = model.step(out[-1], pool, slots)
    return torch.stack(out, 1), torch.stack(seen, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 80), ("batch", 16), ("length", 256), ("serve", 8)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model()
    start = time.time()
    losses, permutation = train(model, args.steps, args.batch, args.length)
    best = -0.9 * math.log(0.9 + 0.1 / model.vocab) - 0.1 * math.log(0.1 / model.vocab)
    print(f"{args.steps} steps in {time.time() - start:.1f} s: loss {losses[0]:.3f} -> {losses[-1]:.3f} "
          f"(the data's own entropy is about {best:.3f})")
    prompts = batch_of(permutation, args.serve, 64, None)[:, :64]
    lengths = torch.randint(1, 65, (args.serve,), device="cuda", dtype=torch.int32)
    tokens, _ = generate(model, prompts, lengths, 32)
    last = prompts[torch.arange(args.serve, device="cuda"), lengths.long() - 1]
    chain = torch.cat([last[:, None], tokens], 1)
    right = (permutation[chain[:, :-1]] == chain[:, 1:]).float().mean().item()
    print(f"{args.serve} prompts of {lengths.min().item()} to {lengths.max().item()} tokens continued by 32: "
          f"{100 * right:.0f} % of the tokens follow the permutation")


if __name__ == "__main__":
    main()
