#!/usr/bin/env python3
"""A hybrid stack served with drafted tokens: Gated DeltaNet layers and attention layers in turn.

Each step takes a few drafted tokens per sequence through the stack at once, checks them against the
target's distributions and keeps the accepted ones and one more:

  attention layer   gdn_kv_append (rotate, quantise, store) then gdn_kv_attn over the 8-bit cache; going
                    back to the kept length needs no call
  GDN layer         gdn_layer from the state before the step; the state moves on by running it over the
                    kept tokens alone
  end of a step     gdn_draft_verify

Weights and prompts are random.  ``python examples/draft_step.py`` prints what each step accepted.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_pre_gb300 as gdn  # noqa: E402

HK, HV, DIM = 2, 6, 128          # GDN layers: key and value heads
HQ, HEADS = 6, 2                 # attention layers: query and kv heads
PAGE, VOCAB, WIDTH = 32, 1000, 256


def _normal(g, *shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _unit(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class GdnLayer:
    """Its state is the convolution's history and the recurrent state of every sequence."""

    def __init__(self, g, n_seq):
        self.d, c = gdn.dims(HK, HV), (2 * HK + HV) * DIM
        self.w_in = _normal(g, WIDTH, c + 2 * HV + HV * DIM, scale=WIDTH ** -0.5)
        self.w_out = _normal(g, HV * DIM, WIDTH, scale=(HV * DIM) ** -0.5)
        self.conv_w = _normal(g, c, 4, scale=0.5, dtype=torch.float32)
        self.A_log = torch.rand(HV, generator=g, device="cuda").mul_(2.0)
        self.dt_bias = _normal(g, HV, scale=0.1, dtype=torch.float32)
        self.gamma = torch.ones(DIM, device="cuda")
        self.hist = torch.zeros((n_seq, c, 3), dtype=torch.float16, device="cuda")
        self.S = torch.zeros((n_seq, HV, DIM, DIM), device="cuda")

    def __call__(self, x, batch):
        cu, T, c = batch["cu"], x.shape[0], self.conv_w.shape[0]
        qkv, a, b, z = (t.contiguous() for t in (x @ self.w_in).split([c, HV, HV, HV * DIM], dim=1))
        y = torch.empty((T, HV, DIM), dtype=torch.float16, device="cuda")
        hist, S = torch.empty_like(self.hist), torch.empty_like(self.S)
        n = cu.shape[0] - 1
        ws = torch.empty(gdn.gdn_layer_workspace_bytes(self.d, n, T), dtype=torch.uint8, device="cuda")
        gdn.gdn_layer(self.d, cu, T, qkv, self.conv_w, self.hist, hist, a, b, z.view(T, HV, DIM), self.A_log,
                      self.dt_bias, self.gamma, self.S, S, False, y, ws)
        if batch["keep"]:
            self.hist, self.S = hist, S
        return y.view(T, -1) @ self.w_out


class AttentionLayer:
    def __init__(self, g, n_seq, most):
        self.w_in = _normal(g, WIDTH, (HQ + 2 * HEADS) * DIM, scale=WIDTH ** -0.5)
        self.w_out = _normal(g, HQ * DIM, WIDTH, scale=(HQ * DIM) ** -0.5)
        n_pages = n_seq * -(-most // PAGE)
        pages = (n_pages, HEADS, PAGE, DIM)
        self.cache = gdn.kv_cache(*(torch.empty(pages, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)),
                                  *(torch.empty((n_pages, HEADS), device="cuda") for _ in range(2)))

    def __call__(self, x, batch):
        T = x.shape[0]
        qkv = (x @ self.w_in).view(T, HQ + 2 * HEADS, DIM)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HEADS], qkv[:, HQ + HEADS:]
        turned, y = (torch.empty((T, HQ, DIM), dtype=torch.float16, device="cuda") for _ in range(2))
        cu, past, table = batch["cu"], batch["past"], batch["table"]
        gdn.gdn_kv_append(self.cache, cu, T, past, table, q, k, v, batch["cos"], batch["sin"], False, turned)
        size = gdn.gdn_kv_attn_workspace_bytes(self.cache, cu.shape[0] - 1, T, HQ, table.shape[1])
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_kv_attn(self.cache, cu, T, past, table, turned, DIM ** -0.5, y, ws)
        return y.view(T, -1) @ self.w_out


class HybridStack:
    """Three GDN layers to one attention layer, the pattern repeated."""

    def __init__(self, n_seq, most, blocks=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n_seq = n_seq
        self.embed = _normal(g, VOCAB, WIDTH)
        self.head = _normal(g, WIDTH, VOCAB, scale=2.0 * WIDTH ** -0.5)
        self.layers = []
        for _ in range(blocks):
            self.layers += [GdnLayer(g, n_seq) for _ in range(3)] + [AttentionLayer(g, n_seq, most)]
        angle = torch.arange(most, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(DIM // 2, device="cuda").double() / (DIM // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        per_seq = -(-most // PAGE)
        self.table = torch.randperm(n_seq * per_seq, generator=g, device="cuda").view(n_seq, per_seq).to(torch.int32)

    def logits(self, tokens, counts, past, keep):
        """Logits after each of the new tokens (a packed batch, counts[s] of sequence s, behind past[s] earlier
        ones); keep: the GDN layers' states move on past them."""
        cu = torch.zeros(self.n_seq + 1, dtype=torch.int32, device="cuda")
        cu[1:] = counts.cumsum(0)
        batch = dict(cu=cu, past=past, table=self.table, cos=self.cos, sin=self.sin, keep=keep)
        x = self.embed[tokens.long()]
        for layer in self.layers:
            x = x + layer(_unit(x), batch)
        return (_unit(x) @ self.head).float()


def draft_step(stack, last, past, drafted, draft_probs, u):
    """One step: `last` [n] the sequences' last kept tokens (not yet in the stack), `drafted` [n, d] with the
    distributions draft_probs [n, d, VOCAB] that they were drawn from.  Returns (accepted [n], next [n]) and
    leaves the stack behind the accepted tokens, `next` the new last ones."""
    n, d = drafted.shape
    tokens = torch.cat((last[:, None], drafted), 1)
    counts = torch.full((n,), d + 1, dtype=torch.int32, device="cuda")
    p = torch.softmax(stack.logits(tokens.reshape(-1), counts, past, keep=False), -1).view(n, d + 1, VOCAB)
    accepted, nxt = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    gdn.gdn_draft_verify(p, draft_probs, drafted, None, u, accepted, nxt)
    kept = accepted + 1
    mine = torch.arange(d + 1, device="cuda")[None] < kept[:, None]
    stack.logits(tokens[mine], kept, past, keep=True)
    return accepted, nxt


def serve(n_seq=4, prompt=40, steps=6, drafts=4, seed=0, say=print):
    """Prompts of different lengths, then `steps` steps; returns (stack, tokens per sequence, past)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = [prompt + 17 * s for s in range(n_seq)]
    stack = HybridStack(n_seq, max(lengths) + steps * (drafts + 1) + drafts + 2, seed=seed)
    texts = [torch.randint(0, VOCAB, (m,), generator=g, device="cuda").tolist() for m in lengths]
    # all of a prompt but its last token
    flat = torch.tensor([t for text in texts for t in text[:-1]], device="cuda")
    counts = torch.tensor([m - 1 for m in lengths], dtype=torch.int32, device="cuda")
    past = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    stack.logits(flat, counts, past, keep=True)
    past = past + counts
    for step in range(steps):
        last = torch.tensor([text[-1] for text in texts], dtype=torch.int32, device="cuda")
        # the draft model of this example: near to uniform
        q = torch.softmax(torch.randn((n_seq, drafts, VOCAB), generator=g, device="cuda") * 0.5, -1)
        drafted = torch.multinomial(q.view(-1, VOCAB), 1, generator=g).view(n_seq, drafts).to(torch.int32)
        u = torch.rand((n_seq, drafts + 1), generator=g, device="cuda")
        accepted, nxt = draft_step(stack, last, past, drafted, q, u)
        for s, (a, t) in enumerate(zip(accepted.tolist(), nxt.tolist())):
            texts[s] += drafted[s, :a].tolist() + [t]
        past = past + accepted + 1
        say(f"step {step}: accepted {accepted.tolist()}, lengths {[len(t) for t in texts]}")
    return stack, texts, past


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--drafts", type=int, default=4)
    args = ap.parse_args()
    serve(n_seq=args.sequences, steps=args.steps, drafts=args.drafts)
