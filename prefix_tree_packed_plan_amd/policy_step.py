"""A policy update on a packed trie of rollouts, end to end on the library's
operators.

    python -m prefix_tree_packed_plan_amd.policy_step [--no-logits]

A small language model -- one recurrent mixer (tree conv + tree gated delta
rule) and one attention layer -- over a prompt with several sampled
completions, each shared token computed once.  Its loss weights every token's
log probability with an advantage and adds an entropy bonus; gradients come
from the library's backward entry points, and the update is plain SGD.  The
program prints the loss of each step.  With --no-logits the log probabilities
and their gradients come straight from the hidden states and the output weight,
no [N, vocab] tensor is kept, and every gradient is bitwise repeatable.
"""
from __future__ import annotations

import argparse
import sys

import torch
from torch.autograd.function import once_differentiable

import prefix_tree_packed_plan_amd as ptp


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table):
        ctx.vocab = table.shape[0]
        ctx.save_for_backward(tokens)
        return ptp.tree_embedding(tokens, table)

    @staticmethod
    @once_differentiable
    def backward(ctx, dx):
        (tokens,) = ctx.saved_tensors
        return None, ptp.tree_embedding_backward(tokens, dx.contiguous(), ctx.vocab)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, plan):
        ctx.plan = plan
        ctx.save_for_backward(x, w)
        return ptp.tree_conv(x, w, plan, act="silu")

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dx, dw, _, _ = ptp.tree_conv_backward(x, w, dy.contiguous(), ctx.plan, act="silu")
        return dx, dw.to(w.dtype), None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, plan):
        o, states = ptp.tree_gdn_scan(q, k, v, g, beta, plan, return_states=True)
        ctx.plan = plan
        ctx.save_for_backward(q, k, v, g, beta, states)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, g, beta, states = ctx.saved_tensors
        dq, dk, dv, dg, db, _ = ptp.tree_gdn_scan_backward(q, k, v, g, beta, do.contiguous(), ctx.plan, states)
        return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype), dg, db, None


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, plan):
        o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
        ctx.plan = plan
        ctx.save_for_backward(q, k, v, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        return (*ptp.tree_attention_backward(*ctx.saved_tensors, do.contiguous(), ctx.plan), None)


class Logprobs(torch.autograd.Function):
    """(logp [N], entropy [N]) of the tokens under logits [N, vocab]."""

    @staticmethod
    def forward(ctx, logits, tokens, plan, temperature):
        r = ptp.tree_logprobs(logits, tokens, plan, temperature=temperature)
        ctx.plan, ctx.temperature = plan, temperature
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        return r.logp, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy):
        logits, tokens, lse, entropy = ctx.saved_tensors
        d = ptp.tree_logprobs_backward(logits, tokens, lse, entropy, dlogp.contiguous(), ctx.plan,
                                       dentropy=dentropy.contiguous(), temperature=ctx.temperature)
        return d, None, None, None


class LinearLogprobs(torch.autograd.Function):
    """Logprobs of the logits hidden @ weight.T, which are not kept."""

    @staticmethod
    def forward(ctx, hidden, weight, tokens, plan, temperature):
        r = ptp.tree_linear_logprobs(hidden, weight, tokens, plan, temperature=temperature)
        ctx.plan, ctx.temperature = plan, temperature
        ctx.save_for_backward(hidden, weight, tokens, r.lse, r.entropy)
        return r.logp, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy):
        hidden, weight, tokens, lse, entropy = ctx.saved_tensors
        return (*ptp.tree_linear_logprobs_backward(hidden, weight, tokens, lse, entropy, dlogp.contiguous(), ctx.plan,
                                                   dentropy=dentropy.contiguous(), temperature=ctx.temperature),
                None, None, None)


class Model:
    """Embedding, recurrent mixer, attention, tied output; `heads` query heads
    over half as many key/value heads of d."""

    def __init__(self, vocab, heads, d, dtype, device, seed=0):
        gen = torch.Generator().manual_seed(seed)
        c = heads * d
        self.heads, self.kv, self.d = heads, max(1, heads // 2), d

        def weight(*shape, std):
            return (torch.randn(shape, generator=gen) * std).to(dtype).to(device).requires_grad_()

        self.embed = weight(vocab, c, std=1.0)
        self.conv = weight(c, 4, std=0.5)
        self.mix = weight(c, 3 * c, std=c ** -0.5)         # q, k, v of the recurrent mixer
        self.gate = weight(c, 2 * heads, std=c ** -0.5)    # its decay and beta
        self.qkv = weight(c, (heads + 2 * self.kv) * d, std=c ** -0.5)
        self.weights = [self.embed, self.conv, self.mix, self.gate, self.qkv]

    def hidden(self, x, plan):
        """The last layer's output for embedded tokens x [N, heads * d]."""
        n, h, d = x.shape[0], self.heads, self.d
        y = Conv.apply(x, self.conv, plan)
        q, k, v = (y @ self.mix).view(n, 3, h, d).unbind(1)
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(x.dtype) for t in (q, k))
        g, beta = (y @ self.gate).float().view(n, 2, h).unbind(1)
        x = x + Scan.apply(q.contiguous(), k.contiguous(), v.contiguous(), -torch.nn.functional.softplus(g),
                           torch.sigmoid(beta), plan).reshape(n, h * d)
        qkv = (x @ self.qkv).view(n, h + 2 * self.kv, d)
        return x + Attention.apply(qkv[:, :h], qkv[:, h:h + self.kv], qkv[:, h + self.kv:], plan).reshape(n, h * d)

    def logits(self, tokens, plan):
        return (self.hidden(self.embed[tokens], plan) @ self.embed.t()) * (self.heads * self.d) ** -0.5

    def logprobs(self, tokens, plan, temperature):
        """(logp, entropy) without logits: their scale goes into the temperature."""
        x = self.hidden(Embedding.apply(tokens, self.embed), plan)
        return LinearLogprobs.apply(x, self.embed, tokens, plan, temperature * (self.heads * self.d) ** 0.5)


def policy_loss(model, tokens, advantage, plan, temperature=1.0, entropy_bonus=0.01, keep_logits=True):
    """-(sum over tokens of advantage x log probability + bonus x entropy) / N,
    each token under its own root-to-token path."""
    if keep_logits:
        logp, entropy = Logprobs.apply(model.logits(tokens, plan), tokens, plan, temperature)
    else:
        logp, entropy = model.logprobs(tokens, plan, temperature)
    return -((advantage * logp).sum() + entropy_bonus * entropy.sum()) / tokens.shape[0]


def policy_step(model, tokens, advantage, plan, lr=0.5, **kw):
    loss = policy_loss(model, tokens, advantage, plan, **kw)
    loss.backward()
    with torch.no_grad():
        for w in model.weights:
            w -= lr * w.grad
            w.grad = None
    return loss.detach()


def rollouts(vocab, device, prompt=160, completions=6, length=90, seed=0):
    """A prompt with completions, one of which forks again; tokens and an
    advantage per token (0 on the prompt)."""
    parents = [-1] + [0] * completions + [completions, completions]
    lens = [prompt] + [length - 7 * i for i in range(completions)] + [17, 30]
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens)
    tokens = torch.randint(0, vocab, (n,), generator=gen).to(device)
    advantage = torch.cat([torch.full((m,), 0.0 if s == 0 else 1.0) for s, m in enumerate(lens)]).to(device)
    return tokens, advantage, ptp.tree_plan(parents, lens, 4)


def main(argv=()):
    ap = argparse.ArgumentParser(description="A policy update on a packed trie of rollouts.")
    ap.add_argument("--no-logits", action="store_true", help="log probabilities without an [N, vocab] tensor")
    keep = not ap.parse_args(argv).no_logits
    device = "cuda:0"
    model = Model(vocab=1003, heads=4, d=64, dtype=torch.bfloat16, device=device)
    tokens, advantage, plan = rollouts(1003, device)
    print(f"{plan.n_tokens} tokens for {plan.stats['path_tokens']} on the paths")
    for i in range(8):
        print(f"step {i}: loss {policy_step(model, tokens, advantage, plan, keep_logits=keep).item():.4f}",
              flush=True)


if __name__ == "__main__":
    main(sys.argv[1:])
