"""Cases of what a server of many requests does around the layers of a hybrid stack: sequences that share
and fork their caches, requests with adapters of their own, and the residual stream between two blocks.

  remap    the page table of the next step from that of the last: rows forked, cut, dropped and grown, a page
           that a growing row shares replaced by a copy of its own, new pages taken from what no row names
  compact  pages renamed so that those in use lie at the front of the pool
  copy     the pages that either of them lists copied, in every layer's cache at once
  norm     a block's output normalised, gated, scaled and added to the residual stream, which is normalised
           for the next block
  adapter  the low-rank adapter of each sequence added to a shared projection's output

``run`` computes a case with elementary torch operations in 32 bits, or, where the module's ``own`` is
true, through the package's entry points.  ``exact`` states the same definitions in 64 bits or, where they
are about whole numbers, on the host.
"""
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
NONE = 1 << 30               # a page that no row names


# ---- cases --------------------------------------------------------------------------------------

def _remap(name, kind, rows, branches, new, past, page, spare):
    """rows sequences of up to `past` tokens; branches: rows made of each; up to `new` tokens of room for
    each; spare: pages in the pool beside those that are needed, in percent (below 0: too few)."""
    return dict(name=name, op="remap", kind=kind, rows=rows, branches=branches, new=new, past=past, page=page,
                spare=spare)


def _compact(name, rows, past, page, filled):
    """filled: percent of the pool's pages that the rows name."""
    return dict(name=name, op="compact", rows=rows, past=past, page=page, filled=filled)


def _copy(name, layers, n_pages, listed_, filled, heads, dim, page, fmt):
    """listed_: entries of the list, of which `filled` percent name pages."""
    return dict(name=name, op="copy", layers=layers, n_pages=n_pages, entries=listed_, filled=filled, heads=heads,
                dim=dim, page=page, fmt=fmt)


def _norm(name, tokens, width, stream, dtype, gate, shared_gate, post, strided):
    return dict(name=name, op="norm", tokens=tokens, width=width, stream=stream, dtype=dtype, gate=gate,
                shared_gate=shared_gate, post=post, strided=strided)


def _adapter(name, n_seq, new, spread, adapters, rank, ragged, d_in, d_out, dtype):
    """ragged: adapters of different ranks up to `rank`."""
    return dict(name=name, op="adapter", n_seq=n_seq, new=new, spread=spread, adapters=adapters, rank=rank,
                ragged=ragged, d_in=d_in, d_out=d_out, dtype=dtype)


def listed():
    return [
        # one decode step of a batch: room for one token a sequence, few of which begin a page
        _remap("remap_step", "step", 64, 1, 1, 8192, 64, 20),
        # 32 long prompts, each sampled eight times: rows share their pages, but for the one that they write
        _remap("remap_branch", "branch", 32, 8, 1, 131072, 64, 10),
        # a small pool after half of its sequences have left
        _compact("compact_small", 64, 8192, 64, 50),
        # a large pool of small pages
        _compact("compact_large", 500, 32768, 16, 70),
        # the pages that 64 forked rows write into, in the attention layers of a 36-layer stack
        _copy("copy_forks", 9, 300, 64, 60, 16, 128, 64, "e4m3"),
        # a compaction's moves
        _copy("copy_moves", 12, 250, 125, 90, 16, 128, 64, "int8"),
        # one decode step of a batch: the smallest call
        _norm("norm_step", 64, 4096, "bf16", "bf16", "none", False, False, False),
        # a prompt; the block's output normalised as well, and gated for each token and channel
        _norm("norm_prompt", 8192, 5120, "bf16", "bf16", "sigmoid", False, True, False),
        # a residual stream in 32 bits, an odd width, one gate for all tokens, the block's output a slice
        _norm("norm_wide", 4001, 7176, "fp32", "fp16", "linear", True, True, True),
        # one decode step of a batch whose sequences have adapters of their own, onto the packed q, k and v channels
        _adapter("adapter_step", 64, 1, "even", 48, 16, False, 4096, 10240, "bf16"),
        # eight prompts of 1 to 4096 tokens
        _adapter("adapter_prompts", 8, 4096, "ragged", 5, 64, False, 4096, 6144, "fp16"),
        # a prompt beside sequences with a few drafted tokens each; ranks of 8 to 128
        _adapter("adapter_mixed", 40, 3001, "mixed", 24, 128, True, 2048, 10240, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _cost(c):
    """What a case holds and moves, in units of the largest listed one of its operator (at most 1)."""
    op = c["op"]
    if op == "remap":
        return max(c["rows"] * c["branches"] * (c["past"] + c["new"]) / c["page"] / (256 * 2049),
                   c["rows"] * (c["past"] + c["branches"] * c["new"]) / c["page"] / 100000)
    if op == "compact":
        return c["rows"] * c["past"] / c["page"] / (500 * 2048) * max(1, 60 / c["filled"])
    if op == "copy":
        return c["layers"] * c["n_pages"] * c["heads"] * c["dim"] * c["page"] / (12 * 250 * 16 * 128 * 64)
    if op == "norm":
        return work(c)["bytes"] / 423e6
    tokens = sum(_lengths(c))
    return max(work(c)["bytes"] / 726e6, tokens * c["rank"] * (c["d_in"] + c["d_out"]) / 1.4e10,
               c["adapters"] * c["rank"] * (c["d_in"] + c["d_out"]) / 4e7)


def draw(rng):
    op = rng.choice(["remap", "compact", "copy", "norm", "norm", "adapter", "adapter", "adapter"])
    if op == "remap":
        kind = rng.choice(["step", "branch", "mixed"])
        c = _remap("", kind, _log(rng, 1, 1000), 1 if kind == "step" else rng.randint(2, 9),
                   rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 4096)]), _log(rng, 10, 131072),
                   rng.choice([16, 32, 64, 128]), rng.choice([-5, 0, 10, 50]))
        shrink = {"rows": 1, "past": 500, "new": 50}
    elif op == "compact":
        c = _compact("", _log(rng, 1, 1000), _log(rng, 10, 131072), rng.choice([16, 32, 64, 128]), rng.randint(5, 100))
        shrink = {"rows": 1, "past": 500}
    elif op == "copy":
        c = _copy("", rng.randint(1, 16), _log(rng, 8, 1000), 1, rng.randint(10, 100), rng.choice([1, 2, 3, 4, 8, 16]),
                  rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"]))
        shrink = {"n_pages": 8, "heads": 1, "layers": 1}
    elif op == "norm":
        c = _norm("", _log(rng, 1, 16384), 8 * _log(rng, 8, 1100), rng.choice(["fp16", "bf16", "fp32"]),
                  rng.choice(["fp16", "bf16"]), rng.choice(["none", "linear", "sigmoid", "silu"]), rng.random() < 0.4,
                  rng.random() < 0.6, rng.random() < 0.3)
        if c["stream"] != "fp32":
            c["dtype"] = c["stream"]
        shrink = {"tokens": 1}
    else:
        kind = rng.choice(["step", "drafts", "prompts", "mixed"])
        n_seq, new, spread = {"step": (_log(rng, 1, 256), 1, "even"),
                              "drafts": (_log(rng, 1, 128), rng.randint(2, 9), "ragged"),
                              "prompts": (_log(rng, 1, 8), _log(rng, 10, 4096), rng.choice(["even", "ragged"])),
                              "mixed": (_log(rng, 2, 64), _log(rng, 10, 4096), "mixed")}[kind]
        c = _adapter("", n_seq, new, spread, _log(rng, 1, 64), rng.choice([8, 16, 24, 32, 64, 64, 128]),
                     rng.random() < 0.4, 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 1280), rng.choice(["fp16", "bf16"]))
        shrink = {"n_seq": 1, "new": 50, "adapters": 4}
    while _cost(c) > 1:
        if max(c[f] / least for f, least in shrink.items()) <= 1:
            shrink = {"d_in": 256, "d_out": 256} if op == "adapter" else {"width": 64} if op == "norm" else shrink
        field = max(shrink, key=lambda f: c[f] / shrink[f])
        c[field] = max(1, int(c[field] * 0.7)) if field not in ("d_in", "d_out", "width") else max(8, int(c[field] * 0.7) // 8 * 8)
    if op == "copy":
        c["entries"] = rng.randint(1, c["n_pages"] // 2)
    del c["name"]
    return c


def _lengths(c):
    """Tokens of each sequence: from the case alone."""
    rng = random.Random("%d/%d/%s" % (c["n_seq"], c["new"], c["spread"]))
    if c["spread"] == "even":
        return [c["new"]] * c["n_seq"]
    if c["spread"] == "mixed":          # one prompt, the others a few tokens each
        return [c["new"]] + [rng.randint(0, 5) for _ in range(c["n_seq"] - 1)]
    new = [rng.randint(0, c["new"]) for _ in range(c["n_seq"])]
    new[0] = c["new"]
    return new


def _choice(c):
    """The adapter of each sequence (some have none) and the adapters' ranks: from the case alone."""
    rng = random.Random("%d/%d/%d" % (c["n_seq"], c["adapters"], c["rank"]))
    ids = [rng.randint(0, c["adapters"] - 1) if rng.random() < 0.95 else -1 for _ in range(c["n_seq"])]
    ids[0] = 0
    ranks = [rng.randint(1, c["rank"] // 8) * 8 if c["ragged"] else c["rank"] for _ in range(c["adapters"])]
    return ids, ranks


def _rows(c):
    """Tokens that each row of the old table holds, and for remap the rows' parents, the tokens that they
    keep and those that they need room for: from the case alone."""
    rng = random.Random("%s/%d/%d/%d" % (c["op"], c["rows"], c["past"], c["page"]))
    held = [max(1, rng.randint(c["past"] // 4, c["past"])) for _ in range(c["rows"])]
    held[-1] = c["past"]
    if c["op"] == "compact":
        return held
    parent, keep, need = [], [], []
    for row in range(c["rows"] * c["branches"]):
        p = row // c["branches"]
        if c["kind"] == "mixed":        # any earlier row, some of its tokens given up; some slots are left empty
            p = rng.randint(0, c["rows"] - 1) if rng.random() < 0.9 else -1
        k = held[p] if p >= 0 else 0
        if c["kind"] == "mixed" and rng.random() < 0.3:
            k = rng.randint(0, k)
        parent.append(p)
        keep.append(k)
        need.append(k + (c["new"] if c["kind"] != "mixed" else rng.choice([0, rng.randint(0, c["new"]), c["new"]])))
    return held, parent, keep, need


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    c = case
    if c["op"] == "remap":
        held, parent, keep, need = _rows(c)
        kept = sum(_pages(k, c["page"]) for k in keep)
        width = max(_pages(x, c["page"]) for x in held + need)
        # the kept entries read, the whole new table written; a mark for each page of the kept entries
        return {"bytes": 4 * (kept + len(parent) * (width + 5)), "flops": kept + len(parent) * width}
    if c["op"] == "compact":
        width = max(_pages(x, c["page"]) for x in _rows(c))
        cells = c["rows"] * width
        return {"bytes": 4 * (2 * cells + 2 * (_pool_pages(c) // 2)), "flops": 2 * cells}
    if c["op"] == "copy":
        moved = c["layers"] * max(1, c["entries"] * c["filled"] // 100)
        page = 2 * c["heads"] * c["page"] * c["dim"] + 8 * c["heads"]
        return {"bytes": 2 * moved * page + 8 * c["entries"], "flops": 0}
    if c["op"] == "norm":
        t, d, x = c["tokens"], c["width"], 4 if c["stream"] == "fp32" else 2
        gates = 0 if c["gate"] == "none" else (1 if c["shared_gate"] else t)
        return {"bytes": t * d * (2 * x + 4) + gates * d * 2 + (2 if c["post"] else 1) * d * 4, "flops": t * d * 12}
    lengths, (ids, ranks) = _lengths(c), _choice(c)
    d = c["d_in"] + c["d_out"]
    mine = [n if a >= 0 else 0 for n, a in zip(lengths, ids)]
    return {"bytes": 2 * (sum(mine) * c["d_in"] + 2 * sum(lengths) * c["d_out"]
                          + sum(ranks[a] for a in {a for n, a in zip(mine, ids) if n}) * d),
            "flops": 2 * sum(n * ranks[a] for n, a in zip(mine, ids)) * d}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pool_pages(c):
    """Pages of a compaction's pool."""
    return max(1, sum(_pages(x, c["page"]) for x in _rows(c)) * 100 // c["filled"])


def _table(c, held, width, order):
    """A table whose entries are pages in the order given.  Every other row shares the first half of the pages
    that it and the row before it hold, as after an earlier fork; returns the pages named too."""
    rows, used = [], 0
    for i, tokens in enumerate(held):
        n, shared = _pages(tokens, c["page"]), 0
        if i % 2:
            shared = min(n, len(rows[-1])) // 2
        rows.append((rows[-1][:shared] if shared else []) + list(range(used, used + n - shared)))
        used += n - shared
    flat = torch.tensor([x for r in rows for x in r], device="cuda", dtype=torch.long)
    count = torch.tensor([len(r) for r in rows], device="cuda")[:, None]
    at = torch.arange(width, device="cuda")[None, :]
    base = torch.cumsum(count, 0) - count
    table = torch.where(at < count, order[flat[(base + at).clamp(max=len(flat) - 1)]], -1)
    return table.to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "remap":
        held, parent, keep, need = _rows(c)
        width = max(_pages(x, c["page"]) for x in held + need)
        old = sum(_pages(x, c["page"]) for x in held)
        more = sum(_pages(n, c["page"]) - k // c["page"] for k, n in zip(keep, need))
        n_pages = max(old, (old + more) * (100 + c["spare"]) // 100)
        table = _table(c, held, width, torch.randperm(n_pages, device="cuda", generator=g))
        return dict(case=c, table=table, parent=torch.tensor(parent, **i32), keep=torch.tensor(keep, **i32),
                    need=torch.tensor(need, **i32), n_pages=n_pages)
    if c["op"] == "compact":
        held, n_pages = _rows(c), _pool_pages(c)
        width = max(_pages(x, c["page"]) for x in held)
        table = _table(c, held, width, torch.randperm(n_pages, device="cuda", generator=g))
        return dict(case=c, table=table, n_pages=n_pages)
    if c["op"] == "copy":
        # normal values in units of a page's scale; a source may be listed more than once, a destination is not
        n, shape = c["n_pages"], (c["n_pages"], c["heads"], c["page"], c["dim"])
        layers = []
        for _ in range(c["layers"]):
            pool = {}
            for x in ("k", "v"):
                codes = torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=g)
                codes = codes.mul_(20).round_().clamp_(-127, 127) if c["fmt"] == "int8" else codes.mul_(64)
                pool[x] = codes.to(CODES[c["fmt"]])
                pool[x + "_scale"] = torch.exp2(torch.randint(-7, -3, shape[:2], device="cuda", generator=g).float())
            layers.append(pool)
        moved = max(1, c["entries"] * c["filled"] // 100)
        order = torch.randperm(n, device="cuda", generator=g)
        source = order[torch.randint(0, n - moved, (moved,), device="cuda", generator=g)]
        place = torch.randperm(c["entries"], device="cuda", generator=g)[:moved]
        copy_from, copy_to = (torch.full((c["entries"],), -1, **i32) for _ in range(2))
        copy_from[place], copy_to[place] = source.to(torch.int32), order[n - moved:].to(torch.int32)
        return dict(case=c, layers=layers, copy_from=copy_from, copy_to=copy_to)
    if c["op"] == "norm":
        t, d, dt = c["tokens"], c["width"], DTYPES[c["dtype"]]

        def normal(*shape, scale=1.0):
            return torch.randn(shape, device="cuda", generator=g) * scale
        # a stream that has grown over some layers, with a few large channels
        channel = torch.exp(normal(d, scale=0.5))
        x = (normal(t, d, scale=3.0) * channel).to(DTYPES[c["stream"]])
        y = normal(t, 2 * d if c["strided"] else d).to(dt)[:, :d]
        gate = None
        if c["gate"] != "none":
            gate = (normal(1 if c["shared_gate"] else t, d) if c["gate"] != "linear" else
                    1 + normal(1 if c["shared_gate"] else t, d, scale=0.2)).to(dt)
            if c["shared_gate"]:
                gate = gate.expand(t, d)
        return dict(case=c, x=x, y=y, gate=gate, post=1 + normal(d, scale=0.1) if c["post"] else None,
                    pre=1 + normal(d, scale=0.1), eps=1e-6, scale=0.5 if c["post"] else 1.0)
    lengths, (ids, ranks) = _lengths(c), _choice(c)
    cu = [0]
    for x in lengths:
        cu.append(cu[-1] + x)
    t, n, r, dt = cu[-1], c["adapters"], c["rank"], DTYPES[c["dtype"]]
    x = torch.randn((t, c["d_in"]), device="cuda", generator=g).to(dt)
    y = torch.randn((t, c["d_out"]), device="cuda", generator=g).to(dt)
    down = (torch.randn((n, r, c["d_in"]), device="cuda", generator=g) * c["d_in"] ** -0.5).to(dt)
    up = (torch.randn((n, r, c["d_out"]), device="cuda", generator=g) * 0.5 * r ** -0.5).to(dt)
    return dict(case=c, cu=torch.tensor(cu, **i32), starts=cu, tokens=t, x=x, y=y, down=down, up=up,
                ids=torch.tensor(ids, **i32), chosen=ids, ranks=torch.tensor(ranks, **i32) if c["ragged"] else None,
                each=ranks, scales=0.5 + 1.5 * torch.rand(n, device="cuda", generator=g))


# ---- the plain form -----------------------------------------------------------------------------

def _free_list(free):
    """Pages of a mask in ascending order, padded with -1."""
    n = free.numel()
    place = torch.where(free, free.long().cumsum(0) - 1, n)
    out = torch.full((n + 1,), -1, dtype=torch.long, device="cuda")
    return out.scatter_(0, place, torch.arange(n, device="cuda"))[:n]


def _remap_plain(s):
    page, n_pages = s["case"]["page"], s["n_pages"]
    table, parent = s["table"], s["parent"].long()
    keep, need = s["keep"].long(), s["need"].long()
    rows, width = parent.numel(), table.shape[1]
    row, at = torch.arange(rows, device="cuda"), torch.arange(width, device="cuda")[None]
    kept = torch.where((parent >= 0) & (parent < table.shape[0]), (keep + page - 1) // page, 0).clamp(0, width)
    end = torch.maximum(kept, ((need + page - 1) // page).clamp(0, width))
    old = table.long()[parent.clamp(0, table.shape[0] - 1)]
    named = (at < kept[:, None]) & (old >= 0) & (old < n_pages)
    # a row that goes on inside its last kept page writes into it
    last = old.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0]
    writes = (need > keep) & (keep < kept * page) & named.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0]
    at_last = writes[:, None] & (at == kept[:, None] - 1)
    owner = torch.full((n_pages + 1,), NONE, dtype=torch.long, device="cuda")
    owner.scatter_reduce_(0, torch.where(named, old, n_pages).flatten(),
                          torch.where(at_last, row[:, None], -1).flatten(), "amin")
    copied = writes & (owner[last.clamp(0, n_pages)] != row)
    wanted = end - kept + copied
    first = wanted.cumsum(0) - wanted
    free = owner[:n_pages] == NONE
    pages = torch.cat((_free_list(free), torch.full(((rows + 1) * (width + 1),), -1, dtype=torch.long, device="cuda")))
    mine = pages[(first + copied)[:, None] + (at - kept[:, None]).clamp(0, width)]
    own_copy = pages[first]
    out = torch.where(named, old, -1)
    out = torch.where(at_last & copied[:, None], own_copy[:, None], out)
    out = torch.where((at >= kept[:, None]) & (at < end[:, None]), mine, out)
    copied &= own_copy >= 0
    total, left = wanted.sum(), free.sum()
    info = torch.stack((n_pages - left + torch.minimum(total, left), (total - left).clamp(min=0)))
    return {"table": out.to(torch.int32), "copy_from": torch.where(copied, last, -1).to(torch.int32),
            "copy_to": torch.where(copied, own_copy, -1).to(torch.int32), "info": info.to(torch.int32)}


def _compact_plain(s):
    table, n = s["table"].long(), s["n_pages"]
    valid = (table >= 0) & (table < n)
    used = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
    used[torch.where(valid, table, n).flatten()] = True
    used = used[:n]
    total = used.sum()
    page = torch.arange(n, device="cuda")
    moved, hole = used & (page >= total), ~used & (page < total)
    sources, holes = _free_list(moved), _free_list(hole)
    name = torch.where(moved, holes[(moved.long().cumsum(0) - 1).clamp(min=0)], page)
    out = torch.where(valid, name[table.clamp(0, n - 1)], -1)
    return {"table": out.to(torch.int32), "copy_from": sources[:n // 2].to(torch.int32),
            "copy_to": holes[:n // 2].to(torch.int32), "info": torch.stack((total, moved.sum())).to(torch.int32)}


def _copy_plain(s):
    there = torch.nonzero((s["copy_from"] >= 0) & (s["copy_to"] >= 0))[:, 0]
    a, b = s["copy_from"].long()[there], s["copy_to"].long()[there]
    for pool in s["layers"]:
        for x in ("k", "v"):
            codes = pool[x].view(torch.uint8)
            codes[b] = codes[a]
            pool[x + "_scale"][b] = pool[x + "_scale"][a]


def _unit(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _norm_plain(s):
    x, u = s["x"].float(), s["y"].float()
    if s["post"] is not None:
        u = _unit(u, s["post"], s["eps"])
    kind = s["case"]["gate"]
    if kind != "none":
        gate = s["gate"].float()
        u = u * (gate if kind == "linear" else torch.sigmoid(gate) if kind == "sigmoid" else gate * torch.sigmoid(gate))
    x = x + s["scale"] * u
    return {"x": x.to(s["x"].dtype), "h": _unit(x, s["pre"], s["eps"]).to(s["y"].dtype)}


def _adapter_plain(s):
    c, out = s["case"], s["y"].float()
    if c["new"] == 1 and c["spread"] == "even":    # one token each: the chosen adapters gathered
        a = s["ids"].long().clamp(min=0)
        h = (s["down"][a].float() @ s["x"].float()[:, :, None])[:, :, 0]
        if s["ranks"] is not None:
            h = torch.where(torch.arange(c["rank"], device="cuda") < s["ranks"][a][:, None], h, 0.0)
        d = (h[:, None, :] @ s["up"][a].float())[:, 0] * s["scales"][a][:, None]
        return torch.where((s["ids"] >= 0)[:, None], out + d, out).to(s["y"].dtype)
    for i, a in enumerate(s["chosen"]):
        lo, hi, r = s["starts"][i], s["starts"][i + 1], s["each"][a]
        if a >= 0 and hi > lo:
            h = s["x"][lo:hi].float() @ s["down"][a, :r].float().T
            out[lo:hi] += s["scales"][a] * (h @ s["up"][a, :r].float())
    return out.to(s["y"].dtype)


# ---- the package's operators --------------------------------------------------------------------

def _scratch(s, size):
    if "workspace" not in s:
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _remap_own(s, gdn):
    rows, width = s["parent"].numel(), s["table"].shape[1]
    ws = _scratch(s, gdn.gdn_kv_remap_workspace_bytes(s["n_pages"], rows, width))
    out, a, b, info = _i32(rows, width), _i32(rows), _i32(rows), _i32(2)
    gdn.gdn_kv_remap(s["table"], s["case"]["page"], s["n_pages"], s["parent"], s["keep"], s["need"], out, a, b, info, ws)
    return {"table": out, "copy_from": a, "copy_to": b, "info": info}


def _compact_own(s, gdn):
    n = s["n_pages"]
    ws = _scratch(s, gdn.gdn_kv_compact_workspace_bytes(n))
    out, a, b, info = _i32(*s["table"].shape), _i32(n // 2), _i32(n // 2), _i32(2)
    gdn.gdn_kv_compact(s["table"], n, out, a, b, info, ws)
    return {"table": out, "copy_from": a, "copy_to": b, "info": info}


def _copy_own(s, gdn):
    if "caches" not in s:
        s["caches"] = gdn.kv_caches([gdn.kv_cache(p["k"], p["v"], p["k_scale"], p["v_scale"]) for p in s["layers"]])
    gdn.gdn_kv_copy(s["caches"], s["copy_from"], s["copy_to"])


def _norm_own(s, gdn):
    x, h = torch.empty_like(s["x"]), torch.empty(s["y"].shape, dtype=s["y"].dtype, device="cuda")
    gdn.gdn_block_norm(s["x"], s["y"], s["gate"], s["case"]["gate"], s["scale"], s["post"], s["pre"], s["eps"], x, h)
    return {"x": x, "h": h}


def _adapter_own(s, gdn):
    c = s["case"]
    ws = _scratch(s, gdn.gdn_adapter_workspace_bytes(c["n_seq"], s["tokens"], c["rank"], c["d_in"]))
    out = torch.empty_like(s["y"])
    gdn.gdn_adapter_add(s["cu"], s["tokens"], s["ids"], s["down"], s["up"], s["ranks"], s["scales"], s["x"], s["y"], out, ws)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        import gated_deltanet_linear_pre_gb300 as gdn
        out = {"remap": _remap_own, "compact": _compact_own, "copy": _copy_own, "norm": _norm_own,
               "adapter": _adapter_own}[op](state, gdn)
    else:
        out = {"remap": _remap_plain, "compact": _compact_plain, "copy": _copy_plain, "norm": _norm_plain,
               "adapter": _adapter_plain}[op](state)
    # a code is a whole number of its page's scale, or a value in units of it
    return state["layers"] if op == "copy" else out


# ---- the definitions in 64 bits, and those about whole numbers on the host ----------------------

def _exact_remap(s):
    page, n_pages = s["case"]["page"], s["n_pages"]
    table, parent = s["table"].tolist(), s["parent"].tolist()
    keep, need, width = s["keep"].tolist(), s["need"].tolist(), s["table"].shape[1]
    rows = []
    for p, k in zip(parent, keep):
        rows.append(table[p][:_pages(k, page)] if 0 <= p < len(table) else [])
    writers, readers = {}, set()
    for i, r in enumerate(rows):
        grows = need[i] > keep[i] and keep[i] % page and r
        for x in r[:-1] if grows else r:
            readers.add(x)
        if grows:
            writers.setdefault(r[-1], []).append(i)
    unnamed = sorted(set(range(n_pages)) - readers - set(writers))
    copy_from, copy_to, given, missing = [-1] * len(rows), [-1] * len(rows), 0, 0

    def take():
        nonlocal given, missing
        if given == len(unnamed):
            missing += 1
            return -1
        given += 1
        return unnamed[given - 1]
    for i, r in enumerate(rows):
        if need[i] > keep[i] and keep[i] % page and r and (r[-1] in readers or writers[r[-1]][0] != i):
            new = take()
            if new >= 0:
                copy_from[i], copy_to[i] = r[-1], new
            r[-1] = new
        while len(r) < _pages(need[i], page):
            r.append(take())
        r += [-1] * (width - len(r))
    i32 = dict(dtype=torch.int32, device="cuda")
    info = [n_pages - len(unnamed) + given, missing]
    return {"table": torch.tensor(rows, **i32), "copy_from": torch.tensor(copy_from, **i32),
            "copy_to": torch.tensor(copy_to, **i32), "info": torch.tensor(info, **i32)}


def _exact_compact(s):
    table, n = s["table"].tolist(), s["n_pages"]
    used = sorted({x for r in table for x in r if x >= 0})
    total = len(used)
    sources = [x for x in used if x >= total]
    taken = set(used)
    holes = [x for x in range(total) if x not in taken]
    name = dict(zip(sources, holes))
    pad = [-1] * (n // 2 - len(sources))
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"table": torch.tensor([[name.get(x, x) for x in r] for r in table], **i32),
            "copy_from": torch.tensor(sources + pad, **i32), "copy_to": torch.tensor(holes + pad, **i32),
            "info": torch.tensor([total, len(sources)], **i32)}


def _exact_copy(s):
    for a, b in zip(s["copy_from"].tolist(), s["copy_to"].tolist()):
        for pool in s["layers"] if a >= 0 and b >= 0 else ():
            for x in ("k", "v"):
                pool[x].view(torch.uint8)[b].copy_(pool[x].view(torch.uint8)[a])
                pool[x + "_scale"][b].copy_(pool[x + "_scale"][a])
    return s["layers"]


def _exact_norm(s):
    """Some rows at a time, norms by the root of a mean of squares."""
    out_x, out_h = (torch.empty(s["x"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, s["x"].shape[0], 1024):
        rows = slice(lo, lo + 1024)
        u = s["y"][rows].double()
        if s["post"] is not None:
            u = u / torch.sqrt(u.square().sum(1, keepdim=True) / u.shape[1] + s["eps"]) * s["post"].double()
        kind = s["case"]["gate"]
        if kind != "none":
            z = s["gate"][rows].double()
            u = u * {"linear": lambda: z, "sigmoid": lambda: 1 / (1 + torch.exp(-z)),
                     "silu": lambda: z / (1 + torch.exp(-z))}[kind]()
        x = s["x"][rows].double() + s["scale"] * u
        out_x[rows] = x
        out_h[rows] = x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + s["eps"]) * s["pre"].double()
    return {"x": out_x, "h": out_h}


def _exact_adapter(s):
    """Adapter by adapter over the tokens of all its sequences, products a thousand tokens at a time."""
    out = s["y"].double()
    seq = torch.tensor([i for i, n in enumerate(_lengths(s["case"])) for _ in range(n)], device="cuda", dtype=torch.long)
    of = s["ids"].long()[seq]
    for a in sorted(set(s["chosen"]) - {-1}):
        at = torch.nonzero(of == a)[:, 0]
        r = s["each"][a]
        down, up, scale = s["down"][a, :r].double(), s["up"][a, :r].double(), float(s["scales"][a])
        for part in at.split(1024):
            h = torch.einsum("td,rd->tr", s["x"][part].double(), down)
            out[part] += scale * torch.einsum("tr,rd->td", h, up)
    return out


def exact(case, seed):
    if case["op"] == "adapter" and work(case)["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    return {"remap": _exact_remap, "compact": _exact_compact, "copy": _exact_copy, "norm": _exact_norm,
            "adapter": _exact_adapter}[case["op"]](s)
