"""Plain 64-bit statements of the paged 8-bit cache, the attention over it and the draft check, written
sequence by sequence in numpy, and the batches that the tests feed to the library.  Nothing here is
shared with the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}   # largest relative rounding error of the type


def values(t):
    """A device tensor's values in 64 bits on the host."""
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def page_table(new, past, page, seed=0, extra=2, width_extra=1):
    """A table whose entries are a shuffled choice of the pool's pages; entries behind a sequence's end are
    out of range.  Returns (table int32 [n, width], n_pages)."""
    rng = np.random.default_rng(seed)
    held = [max(0, -(-max(0, a + b) // page)) for a, b in zip(new, past)]
    n_pages = max(1, sum(held)) + extra
    ids = rng.permutation(n_pages)
    table = np.full((len(new), max(held + [0]) + width_extra), -1, np.int32)
    table[:, -1] = n_pages + 5
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        at += h
    return table, n_pages


def rotate(x, pos, cos, sin, interleaved):
    """x [T, h, d] at positions pos [T], float64."""
    y = x.copy()
    if cos is None:
        return y
    half = cos.shape[1]
    c = cos[np.clip(pos, 0, len(cos) - 1)][:, None, :]
    s = sin[np.clip(pos, 0, len(cos) - 1)][:, None, :]
    ia, ib = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def positions(cu, past):
    return np.concatenate([past[s] + np.arange(cu[s + 1] - cu[s]) for s in range(len(past))] + [np.zeros(0, int)]).astype(int)


def dense(pages, scale, table, s, held, page):
    """Values [held, heads, d] of sequence s and whether each position has a page."""
    n_pages, heads, _, d = pages.shape
    out = np.zeros((held, heads, d))
    there = np.zeros(held, bool)
    for j in range(held):
        at = j // page
        if at < table.shape[1] and 0 <= table[s, at] < n_pages:
            pg = table[s, at]
            out[j] = pages[pg, :, j % page] * scale[pg][:, None]
            there[j] = True
    return out, there


def attention(q, k_pages, v_pages, k_scale, v_scale, table, cu, past, page, softmax_scale):
    """(y, W, X): the outputs, sum_j w_j |v_j| and the largest sum |q||k| scale, all in 64 bits."""
    T, hq, d = q.shape
    heads = k_pages.shape[1]
    group = hq // heads
    y, wabs, xabs = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq, 1))
    for s in range(len(past)):
        n = cu[s + 1] - cu[s]
        held = max(0, past[s] + n)
        if n == 0 or held == 0:
            continue
        k, there = dense(k_pages, k_scale, table, s, held, page)
        v, _ = dense(v_pages, v_scale, table, s, held, page)
        for i in range(n):
            see = min(held, past[s] + i + 1)
            on = there[:max(see, 0)]
            if not on.any():
                continue
            kk, vv = k[:see][on], v[:see][on]
            for h in range(hq):
                x = (kk[:, h // group] @ q[cu[s] + i, h]) * softmax_scale
                w = np.exp(x - x.max())
                w /= w.sum()
                y[cu[s] + i, h] = w @ vv[:, h // group]
                wabs[cu[s] + i, h] = w @ np.abs(vv[:, h // group])
                xabs[cu[s] + i, h] = (np.abs(kk[:, h // group]) @ np.abs(q[cu[s] + i, h])).max() * abs(softmax_scale)
    return y, wabs, xabs


def attention_bound(y, wabs, xabs, dtype):
    """Largest error that the stated roundings allow: the output type's; the weights' to fp16 (2^-11 with the
    sum's and the exponential's own errors); the scores' fp32 sums of up to 128 products (16 accumulation
    steps of at most 2^-23 each, and the scaling's 2^-22), which enter the weights through exp (twice: the
    normalising sum has the same error); the least fp16 step of a small output."""
    score = xabs * 2.0 ** -18
    return UNIT[dtype] * np.abs(y) + wabs * (2.0 ** -11 + 2.0 * score) + 2.0 ** -24


def verify(p, q, draft, count, u):
    """(accepted, next) of one sequence: p [d + 1, V], q [d, V] float32 arrays; whole-number weights."""
    d, V = len(draft), p.shape[1]
    count = min(max(count, 0), d)
    a = 0
    while a < count:
        x = draft[a]
        if not (0 <= x < V and np.float32(u[a]) * q[a, x] < p[a, x]):
            break
        a += 1
    rows = [(p[a] - q[a]).astype(np.float32), p[a]] if a < count else [p[a]]
    for r in rows:
        with np.errstate(invalid="ignore"):
            x = np.where(np.isnan(r), np.float32(0), np.clip(r, 0, 1)).astype(np.float64)
        w = [int(z) for z in np.floor(x * 2.0 ** 43)]
        total = sum(w)
        if total > 0:
            limit = min(int(np.floor(np.float64(np.float32(u[d])) * np.float64(total))), total - 1)
            run = 0
            for i, z in enumerate(w):
                run += z
                if run > limit:
                    return a, i
    return a, -1
