#!/usr/bin/env python3
"""A hybrid stack served with drafted tokens: Gated DeltaNet layers and attention layers in turn.

Each step takes a few drafted tokens per sequence through the stack at once, checks them against the
target's distributions and keeps the accepted ones and one more:

  attention layer   gdn_kv_append (rotate, quantise, store) then gdn_kv_attn over the 8-bit cache; going
                    back to the kept length needs no call
  GDN layer         gdn_layer from the state before the step; the state moves on by running it over the
                    kept tokens alone
  end of a step     gdn_draft_verify

With --branches, each prompt is sampled several times: the sequences share the prompt's pages of every attention
layer's cache (gdn_kv_remap, which also finds room for each step's tokens, and gdn_kv_copy for the page that a branch
writes into); the GDN layers' states are copied.  With --adapters, each sequence has a low-rank adapter of its own on
the layers' projections to q, k and v (gdn_adapter_add).  Either way the residual stream goes through gdn_block_norm.

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
RANK = 8                         # of the adapters


def _normal(g, *shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _unit(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


def _adapt(layer, x, y, batch):
    """The sequences' adapters added to y, what the layer's projection makes of x."""
    if layer.adapters is not None:
        down, up, scales = layer.adapters
        cu, T = batch["cu"], x.shape[0]
        size = gdn.gdn_adapter_workspace_bytes(cu.shape[0] - 1, T, RANK, WIDTH)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_adapter_add(cu, T, batch["ids"], down, up, None, scales, x, y, y, ws)
    return y


class GdnLayer:
    """Its state is the convolution's history and the recurrent state of every sequence."""

    adapters = None

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
        _adapt(self, x, qkv, batch)
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
    adapters = None

    def __init__(self, g, n_seq, most):
        self.w_in = _normal(g, WIDTH, (HQ + 2 * HEADS) * DIM, scale=WIDTH ** -0.5)
        self.w_out = _normal(g, HQ * DIM, WIDTH, scale=(HQ * DIM) ** -0.5)
        n_pages = n_seq * -(-most // PAGE)
        pages = (n_pages, HEADS, PAGE, DIM)
        self.cache = gdn.kv_cache(*(torch.empty(pages, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)),
                                  *(torch.empty((n_pages, HEADS), device="cuda") for _ in range(2)))

    def __call__(self, x, batch):
        T = x.shape[0]
        qkv = _adapt(self, x, x @ self.w_in, batch).view(T, HQ + 2 * HEADS, DIM)
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

    def __init__(self, n_seq, most, blocks=2, seed=0, rows=None, adapters=0):
        """rows: sequences that the caches have pages for, where they come to be more than n_seq; the page table is
        then gdn_kv_remap's.  adapters: how many there are; sequence s begins with adapter s % adapters."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n_seq = n_seq
        self.fused = rows is not None or adapters > 0
        self.embed = _normal(g, VOCAB, WIDTH)
        self.head = _normal(g, WIDTH, VOCAB, scale=2.0 * WIDTH ** -0.5)
        self.layers = []
        for _ in range(blocks):
            self.layers += [GdnLayer(g, n_seq) for _ in range(3)] + [AttentionLayer(g, rows or n_seq, most)]
        angle = torch.arange(most, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(DIM // 2, device="cuda").double() / (DIM // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        per_seq = -(-most // PAGE)
        self.n_pages = (rows or n_seq) * per_seq
        self.table = torch.randperm(n_seq * per_seq, generator=g, device="cuda").view(n_seq, per_seq).to(torch.int32)
        self.remapped = rows is not None
        if self.remapped:
            self.table.fill_(-1)
            self.caches = gdn.kv_caches([layer.cache for layer in self.layers if isinstance(layer, AttentionLayer)])
        if adapters:
            self.ids = torch.arange(n_seq, dtype=torch.int32, device="cuda") % adapters
            for layer in self.layers:
                out = layer.conv_w.shape[0] if isinstance(layer, GdnLayer) else layer.w_in.shape[1]
                layer.adapters = (_normal(g, adapters, RANK, WIDTH, scale=WIDTH ** -0.5),
                                  _normal(g, adapters, RANK, out, scale=0.5 * RANK ** -0.5), torch.ones(adapters, device="cuda"))
        self.ones = torch.ones(WIDTH, device="cuda")

    def remap(self, parent, keep, need):
        """The sequences become rows of the ones there are: row r goes on from the first keep[r] tokens of sequence
        parent[r], with room for need[r].  Returns the pages in use."""
        rows, width = parent.shape[0], self.table.shape[1]
        out, i32 = torch.empty((rows, width), dtype=torch.int32, device="cuda"), dict(dtype=torch.int32, device="cuda")
        copy_from, copy_to, info = torch.empty(rows, **i32), torch.empty(rows, **i32), torch.empty(2, **i32)
        ws = torch.empty(gdn.gdn_kv_remap_workspace_bytes(self.n_pages, rows, width), dtype=torch.uint8, device="cuda")
        gdn.gdn_kv_remap(self.table, PAGE, self.n_pages, parent, keep, need, out, copy_from, copy_to, info, ws)
        gdn.gdn_kv_copy(self.caches, copy_from, copy_to)
        self.table = out
        return info

    def branch(self, parent, past):
        """Sequences parent[r] go on side by side from what they hold."""
        self.remap(parent, past, past)
        for layer in self.layers:
            if isinstance(layer, GdnLayer):
                layer.hist, layer.S = layer.hist[parent.long()], layer.S[parent.long()]
        if any(layer.adapters is not None for layer in self.layers):
            self.ids = self.ids[parent.long()]
        self.n_seq = parent.shape[0]

    def logits(self, tokens, counts, past, keep):
        """Logits after each of the new tokens (a packed batch, counts[s] of sequence s, behind past[s] earlier
        ones); keep: the GDN layers' states move on past them."""
        cu = torch.zeros(self.n_seq + 1, dtype=torch.int32, device="cuda")
        cu[1:] = counts.cumsum(0)
        if self.remapped:
            rows = torch.arange(self.n_seq, dtype=torch.int32, device="cuda")
            self.remap(rows, past, past + counts)
        batch = dict(cu=cu, past=past, table=self.table, cos=self.cos, sin=self.sin, keep=keep, ids=getattr(self, "ids", None))
        x = self.embed[tokens.long()]
        if self.fused:
            h = torch.empty_like(x)
            gdn.gdn_block_norm(x, None, None, "none", 1.0, None, self.ones, 1e-6, None, h)
            for layer in self.layers:
                y = layer(h, batch)
                gdn.gdn_block_norm(x, y, None, "none", 1.0, None, self.ones, 1e-6, x, h)
            return (h @ self.head).float()
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


def serve(n_seq=4, prompt=40, steps=6, drafts=4, seed=0, say=print, branches=1, adapters=0):
    """Prompts of different lengths, each sampled `branches` times, then `steps` steps; returns (stack, tokens per
    sequence, past)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = [prompt + 17 * s for s in range(n_seq)]
    stack = HybridStack(n_seq, max(lengths) + steps * (drafts + 1) + drafts + 2, seed=seed,
                        rows=n_seq * branches if branches > 1 else None, adapters=adapters)
    texts = [torch.randint(0, VOCAB, (m,), generator=g, device="cuda").tolist() for m in lengths]
    # all of a prompt but its last token
    flat = torch.tensor([t for text in texts for t in text[:-1]], device="cuda")
    counts = torch.tensor([m - 1 for m in lengths], dtype=torch.int32, device="cuda")
    past = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    stack.logits(flat, counts, past, keep=True)
    past = past + counts
    if branches > 1:
        parent = torch.arange(n_seq, dtype=torch.int32, device="cuda").repeat_interleave(branches)
        past = past[parent.long()]
        stack.branch(parent, past)
        texts = [list(texts[p]) for p in parent.tolist()]
        n_seq = n_seq * branches
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
    ap.add_argument("--branches", type=int, default=1, help="samples of each prompt")
    ap.add_argument("--adapters", type=int, default=0, help="low-rank adapters, dealt out to the sequences")
    args = ap.parse_args()
    serve(n_seq=args.sequences, steps=args.steps, drafts=args.drafts, branches=args.branches, adapters=args.adapters)
