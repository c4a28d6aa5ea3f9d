"""Speculative decoding end to end on a small random model: the target's
forward pass over a paged cache, the verify step, and a drafter that learns
from the target's top logits while it drafts.

Per round and sequence:

  draft    gamma tokens from a bigram drafter
  append   keys and values of the chunk (the last token and its drafts),
           rotated by position, into the paged cache     api.kv_append
  attend   the chunk over the cache                      api.paged_attention
  verify   the drafts against the target's logits        api.verify_linear
  commit   n accepted drafts: the cache's length grows by n + 1; what the
           rejected ones left behind is overwritten by the next round
  distill  the target's top logits of every row of the chunk
           (api.fanout_topk) train the drafter           api.distill_topk_step

    python examples/speculative_round.py --rounds 80
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                ".."))
from speculative_decoding_verification_temperature_gb300 import api  # noqa


class Target:
    """One attention layer over a paged cache, between random embeddings."""

    def __init__(self, V, q_heads, heads, dim, B, max_len, page, gen):
        def randn(*shape, by=1.0):
            return (torch.randn(shape, generator=gen, device="cuda") * by).to(
                torch.bfloat16)
        d = q_heads * dim
        self.embed = randn(V, d)
        self.qkv = randn(d, (q_heads + 2 * heads) * dim, by=1.5 * d ** -0.5)
        self.out = randn(d, V, by=3 * d ** -0.5)
        self.q_heads, self.heads, self.dim = q_heads, heads, dim
        pages = -(-max_len // page)
        self.cache = api.PagedKV(
            randn(B * pages, page, heads, dim),
            randn(B * pages, page, heads, dim),
            torch.randperm(B * pages, generator=gen, device="cuda").to(
                torch.int32).view(B, pages))
        f = 10000.0 ** (-torch.arange(dim // 2, device="cuda") * 2.0 / dim)
        a = torch.arange(max_len, device="cuda")[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1)
        self.workspace = api.Workspace()

    def logits(self, tokens, q_start, kv_len, max_q, status):
        """fp32 logits of packed tokens, whose chunks end at kv_len."""
        x = self.embed[tokens]
        h = self.q_heads
        qkv = (x @ self.qkv).view(len(tokens), h + 2 * self.heads, self.dim)
        q = api.kv_append(self.cache, qkv[:, h:h + self.heads],
                          qkv[:, h + self.heads:], q_start, kv_len,
                          q=qkv[:, :h], cos_sin=self.cos_sin, status=status)
        o = api.paged_attention(q, self.cache, q_start, kv_len, max_q=max_q,
                                workspace=self.workspace,
                                status=status)["out"]
        return ((x + o.flatten(1)) @ self.out).float()


class Drafter:
    """A bigram model: logits of the next token from the last one alone."""

    def __init__(self, V, d, gen):
        self.embed = torch.randn(V, d, generator=gen, device="cuda") * \
            d ** -0.5
        self.head = torch.zeros(V, d, device="cuda")

    def logits(self, tokens):
        return self.embed[tokens] @ self.head.T

    def learn(self, tokens, grad, rate):
        self.head -= rate * (grad.T @ self.embed[tokens])


def main(rounds=80, B=32, gamma=4, V=256, T=1.0, top=64, rate=200.0, seed=0,
         verbose=True):
    """Returns per-round lists: mean accepted drafts, mean loss; and the
    status word (0: nothing was out of order)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    prompt, G = 20, gamma + 1
    target = Target(V, 8, 2, 64, B, prompt + (rounds + 1) * G, 16, gen)
    drafter = Drafter(V, 256, gen)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    # the prompts, all but their last token
    tokens = torch.randint(V, (B, prompt), generator=gen, device="cuda")
    start = torch.arange(0, B * (prompt - 1) + 1, prompt - 1, **i32)
    length = torch.full((B,), prompt - 1, **i32)
    target.logits(tokens[:, :-1].flatten(), start, length, prompt - 1, status)

    last = tokens[:, -1]
    start = torch.arange(0, B * G + 1, G, **i32)
    weight = torch.full((B * G,), 1.0 / (B * G), device="cuda")
    accepted, losses = [], []
    for _ in range(rounds):
        draft, rows, x = [], [], last
        for _ in range(gamma):
            z = drafter.logits(x)
            rows.append(z)
            x = torch.multinomial(torch.softmax(z / T, 1), 1,
                                  generator=gen)[:, 0]
            draft.append(x)
        drafts = torch.stack(draft, 1)
        chunk = torch.cat([last[:, None], drafts], 1)
        z = target.logits(chunk.flatten(), start, length + G, G, status)
        u = torch.rand(B, G, generator=gen, device="cuda") * 0.999 + 5e-4
        v = api.verify_linear(z.view(B, G, V), torch.stack(rows, 1),
                              drafts.to(torch.int32), u, T, status=status)
        n = v["n"]
        # the next chunk starts at the correction or bonus token, whose own
        # key is not in the cache yet: n drafts and the old last token are
        last = v["tokens"].gather(1, n.long()[:, None])[:, 0].long()
        length = length + n + 1
        fan = api.fanout_topk(z.view(B, G, V), [top] * G, want_logit=True,
                              status=status)
        step = api.distill_topk_step(
            drafter.logits(chunk.flatten()), fan["logit"].view(-1, top),
            fan["tokens"].view(-1, top), weight, T, status=status)
        drafter.learn(chunk.flatten(), step["grad"], rate)
        accepted.append(n.float().mean())
        losses.append(step["loss"].mean())
    accepted = torch.stack(accepted).tolist()
    losses = torch.stack(losses).tolist()
    if verbose:
        for i in range(0, rounds, max(1, rounds // 10)):
            print("round %3d: %.2f of %d drafts accepted, loss %.3f" %
                  (i, accepted[i], gamma, losses[i]))
        print("status", int(status.item()))
    return accepted, losses, int(status.item())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--rounds", type=int, default=80)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--gamma", type=int, default=4)
    args = ap.parse_args()
    main(args.rounds, args.batch, args.gamma)
