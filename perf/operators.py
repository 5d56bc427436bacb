"""Cases of the attention layers that sit between Gated DeltaNet layers in a hybrid stack, when it
serves prompts, single tokens and drafted tokens:

  append   new keys and values rotated by their positions, quantised to 8 bits and stored in a paged
           cache (one power-of-two scale per page and head); queries rotated in the same call
  attn     causal attention of the new tokens over that cache
  verify   drafted tokens checked against the target's probabilities from given random numbers

``run`` computes a case with elementary torch operations in 32 bits, or, where the module's ``own`` is
true, through the package's entry points.  ``exact`` states the same definitions in 64 bits.
"""
import random

import torch

own = False

INT8, E4M3 = "int8", "e4m3"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {INT8: torch.int8, E4M3: torch.float8_e4m3fn}
POSITIONS = 1 << 18          # rows a rotation table may have
WEIGHT_BITS = 43             # sampling weights are whole multiples of 2^-43


# ---- cases --------------------------------------------------------------------------------------

def _append(name, n_seq, new, past, spread, hq, hkv, dim, page, fmt, dtype, rot, interleaved):
    return dict(name=name, op="append", n_seq=n_seq, new=new, past=past, spread=spread, hq=hq, hkv=hkv, dim=dim,
                page=page, fmt=fmt, dtype=dtype, rot=rot, interleaved=interleaved)


def _attn(name, n_seq, new, past, spread, hq, hkv, dim, page, fmt, dtype):
    return dict(name=name, op="attn", n_seq=n_seq, new=new, past=past, spread=spread, hq=hq, hkv=hkv, dim=dim,
                page=page, fmt=fmt, dtype=dtype)


def _verify(name, n_seq, drafts, vocab, spread):
    return dict(name=name, op="verify", n_seq=n_seq, drafts=drafts, vocab=vocab, spread=spread)


def listed():
    return [
        # one decode step of a batch: one token per sequence, each at its own place in a page
        _append("append_step", 64, 1, 2047, "ragged", 32, 8, 128, 64, E4M3, "bf16", 128, False),
        # a few drafted tokens per sequence, small pages, neighbouring channels rotated in part of the head
        _append("append_drafts", 37, 5, 1000, "ragged", 48, 16, 128, 16, INT8, "fp16", 64, True),
        # eight prompts of 1 to 4096 tokens, as the package's variable-length batch
        _append("append_prompts", 8, 4096, 0, "ragged", 48, 16, 128, 64, E4M3, "fp16", 128, False),
        # the smallest call: one token of one short sequence, where latency counts
        _attn("attn_step_one", 1, 1, 300, "even", 48, 16, 128, 16, INT8, "fp16"),
        # one decode step of a batch with caches of any length up to 8192
        _attn("attn_step_batch", 64, 1, 8191, "ragged", 32, 4, 128, 64, E4M3, "bf16"),
        # single tokens over long contexts: few rows, a long axis
        _attn("attn_step_long", 3, 1, 131000, "even", 16, 4, 64, 128, INT8, "bf16"),
        # drafted tokens of a batch attend together
        _attn("attn_drafts", 37, 6, 4099, "ragged", 48, 16, 128, 32, E4M3, "fp16"),
        # the package's prompt length from an empty cache
        _attn("attn_prompt", 1, 2048, 0, "even", 48, 16, 128, 64, E4M3, "fp16"),
        # a long prompt's later chunk beside sequences that decode: the largest
        _attn("attn_chunk_mixed", 4, 4001, 16500, "mixed", 32, 4, 128, 64, INT8, "bf16"),
        # one sequence, a small vocabulary
        _verify("verify_one", 1, 4, 32768, "even"),
        # a batch whose sequences hold different numbers of drafts; rows of odd length
        _verify("verify_ragged", 64, 5, 100003, "ragged"),
        # a large batch and vocabulary
        _verify("verify_batch", 256, 7, 131072, "ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _cost(c):
    """What a case's plain form holds and computes, in units of the largest listed one (at most 1)."""
    if c["op"] == "verify":
        return c["n_seq"] * (2 * c["drafts"] + 1) * c["vocab"] / (256 * 15 * 131072)
    new, past = _lengths(c)
    pool = sum(-(-(n + p) // c["page"]) * c["page"] for n, p in zip(new, past)) * c["hkv"] * c["dim"] * 2
    if c["op"] == "append":
        return max(pool / 2e9, sum(new) / 28000)
    most_new, most = max(new), max(n + p for n, p in zip(new, past))
    scores = c["n_seq"] * c["hq"] * most_new * most
    gathered = c["n_seq"] * c["hkv"] * most * c["dim"]
    return max(scores / (4 * 32 * 4001 * 20501), gathered / 1.5e9, work(c)["flops"] / 1.2e12)


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "verify"])
    if op == "verify":
        c = _verify("", _log(rng, 1, 256), rng.randint(1, 8), _log(rng, 1000, 131072), rng.choice(["even", "ragged"]))
        shrink = ("n_seq", "vocab")
    else:
        hkv = rng.choice([1, 2, 4, 8, 16])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16]) if hkv < 8 else hkv * rng.choice([1, 2, 3, 4, 5])
        dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
        fmt, dtype = rng.choice([INT8, E4M3]), rng.choice(["fp16", "bf16"])
        kind = rng.choice(["step", "drafts", "prompt"])
        spread = rng.choice(["even", "ragged", "mixed"])
        if kind == "step":
            n_seq, new, past = _log(rng, 1, 256), 1, _log(rng, 1, 131072)
        elif kind == "drafts":
            n_seq, new, past = _log(rng, 1, 128), rng.randint(2, 9), _log(rng, 1, 32768)
        else:
            n_seq, new, past = _log(rng, 1, 8), _log(rng, 10, 4096), rng.choice([0, _log(rng, 1, 16384)])
        if op == "append":
            c = _append("", n_seq, new, past, spread, hq, hkv, dim, page, fmt, dtype,
                        rng.choice([0, dim // 4, dim // 2, dim, dim]), rng.random() < 0.5)
        else:
            c = _attn("", n_seq, new, past, spread, hq, hkv, dim, page, fmt, dtype)
        shrink = ("n_seq", "past", "new")
    while _cost(c) > 1:
        field = max(shrink, key=lambda f: c[f] / {"n_seq": 1, "vocab": 1000, "past": 500, "new": 500}[f])
        c[field] = max(1, int(c[field] * 0.7))
    del c["name"]
    return c


def _lengths(c):
    """New tokens and tokens already in the cache, per sequence: from the case alone."""
    rng = random.Random("%d/%d/%d/%s" % (c["n_seq"], c["new"], c["past"], c["spread"]))
    n = c["n_seq"]
    if c["spread"] == "even":
        return [c["new"]] * n, [c["past"]] * n
    past = [rng.randint(0, c["past"]) for _ in range(n)]
    if c["spread"] == "mixed":          # one sequence brings many tokens, the others one each
        past[0] = c["past"]
        return [c["new"]] + [1] * (n - 1), past
    new = [rng.randint(0, c["new"]) if c["new"] > 1 else 1 for _ in range(n)]
    new[0], past[-1] = c["new"], c["past"]
    return new, past


def work(case):
    c = case
    if c["op"] == "verify":
        # the p and q rows of one position per sequence, read once (a sequence that takes all its drafts has no
        # q row there: that depends on the random numbers)
        rows = c["n_seq"] * c["vocab"]
        return {"bytes": rows * 8 + c["n_seq"] * (c["drafts"] * 16 + 20), "flops": rows * 4}
    new, past = _lengths(c)
    hq, hkv, dim, tokens = c["hq"], c["hkv"], c["dim"], sum(new)
    if c["op"] == "append":
        pages = sum((n + p - 1) // c["page"] - p // c["page"] + 1 for n, p in zip(new, past) if n)
        rows = tokens * (2 * hq * dim * 2 + 2 * hkv * dim * (2 + 1))
        return {"bytes": rows + 2 * pages * hkv * 4 + tokens * c["rot"] * 4,
                "flops": tokens * ((hq + hkv) * c["rot"] * 3 + 2 * hkv * dim * 3)}
    held = sum(n + p for n, p in zip(new, past) if n)
    pages = sum(-(-(n + p) // c["page"]) for n, p in zip(new, past) if n)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return {"bytes": 2 * held * hkv * dim + 2 * pages * hkv * 4 + 2 * tokens * hq * dim * 2,
            "flops": 4 * dim * hq * pairs}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _batch(c, g):
    """Offsets, lengths and a page table whose entries are a random choice of the pool's pages."""
    new, past = _lengths(c)
    page, n = c["page"], c["n_seq"]
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    held = [-(-(a + b) // page) for a, b in zip(new, past)]
    width, n_pages = max(1, max(held)), max(1, sum(held))
    count = torch.tensor(held, device="cuda")[:, None]
    at = torch.arange(width, device="cuda")[None, :]
    order = torch.randperm(n_pages, device="cuda", generator=g)
    base = torch.cumsum(count, 0) - count
    table = torch.where(at < count, order[(base + at).clamp(max=n_pages - 1)], -1).to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(cu=torch.tensor(cu, **i32), past=torch.tensor(past, **i32), table=table.contiguous(), tokens=cu[-1],
                n_pages=n_pages, most_new=max(new), most=max(a + b for a, b in zip(new, past)))


def _pool(c, n_pages, g):
    """Codes and scales as a cache holds them after earlier calls: normal values, the scale of a page and
    head the power of two that its largest value needs."""
    shape = (n_pages, c["hkv"], c["page"], c["dim"])
    codes, scales = [], []
    for _ in range(2):
        x = torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=g)
        spread = torch.randint(-1, 2, (n_pages, c["hkv"]), device="cuda", generator=g).float()
        if c["fmt"] == INT8:
            codes.append((x * 20).round_().clamp_(-127, 127).to(torch.int8))
            scales.append(torch.exp2(spread - 4))
        else:
            codes.append((x * 64).to(torch.float8_e4m3fn))
            scales.append(torch.exp2(spread - 6))
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1])


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "verify":
        n, k, vocab = c["n_seq"], c["drafts"], c["vocab"]
        draft_logits = torch.randn((n, k, vocab), device="cuda", generator=g).mul_(2.5)
        logits = torch.randn((n, k + 1, vocab), device="cuda", generator=g).mul_(1.0)
        logits[:, :k] += draft_logits
        q = torch.softmax(draft_logits, -1)
        p = torch.softmax(logits, -1)
        del logits, draft_logits
        draft = torch.multinomial(q.view(n * k, vocab), 1, generator=g).view(n, k).to(torch.int32)
        if c["spread"] == "ragged":
            count = torch.randint(0, k + 1, (n,), device="cuda", generator=g).to(torch.int32)
        else:
            count = torch.full((n,), k, dtype=torch.int32, device="cuda")
        u = torch.rand((n, k + 1), device="cuda", generator=g)
        return dict(case=c, p=p, q=q, draft=draft, count=count, u=u)
    s = _batch(c, g)
    dt = DTYPES[c["dtype"]]
    # one page more than the tables name: the plain form sends what it must not store there
    s |= _pool(c, s["n_pages"] + 1, g)
    t, hq, hkv, dim = s["tokens"], c["hq"], c["hkv"], c["dim"]
    if c["op"] == "append":
        # q, k and v as the layer's projection leaves them: side by side in one row per token
        qkv = torch.randn((t, hq + 2 * hkv, dim), device="cuda", generator=g).to(dt)
        s |= dict(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:])
        if c["rot"]:
            half = c["rot"] // 2
            freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
            angle = torch.arange(s["most"], device="cuda", dtype=torch.float64)[:, None] * freq
            s |= dict(cos=angle.cos().float(), sin=angle.sin().float())
        else:
            s |= dict(cos=None, sin=None)
    else:
        s["q"] = (torch.randn((t, hq, dim), device="cuda", generator=g) * 1.5).to(dt)
    return dict(case=c, **s)


# ---- the plain form -----------------------------------------------------------------------------

def _rotate(x, pos, cos, sin, interleaved):
    if cos is None:
        return x
    half = cos.shape[1]
    c, s = cos[pos][:, None, :], sin[pos][:, None, :]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _token_places(s):
    tok = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:], tok, right=True)
    return tok, seq, s["past"].long()[seq] + tok - s["cu"].long()[seq]


def _scale_for(amax, fmt):
    """The smallest power of two that brings `amax` into the format's range (at least 2^-100; 0 for 0;
    NaN where a value is not finite)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 127 / 128, e - 7, e - 6) if fmt == INT8 else torch.where(m <= 0.875, e - 9, e - 8)
    scale = torch.ldexp(torch.ones_like(amax), e.clamp(min=-100))
    scale = torch.where(amax == 0, torch.zeros_like(amax), scale)
    return torch.where(torch.isfinite(amax), scale, torch.full_like(amax, float("nan")))


def _encode(x, scale, fmt):
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    return y.round().to(torch.int8) if fmt == INT8 else y.to(torch.float8_e4m3fn)


def _rows(codes, at):
    return codes.view(torch.uint8)[at].view(codes.dtype)


def _append_plain(s):
    c = s["case"]
    page, fmt = c["page"], c["fmt"]
    cu, past, table = s["cu"].long(), s["past"].long(), s["table"].long()
    tok, seq, pos = _token_places(s)
    q = _rotate(s["q"].float(), pos, s["cos"], s["sin"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k_new"].float(), pos, s["cos"], s["sin"], c["interleaved"])
    v = s["v_new"].float()
    # one slot for each page that a sequence may touch; slots that touch none go to the spare page
    base = cu // page + 2 * torch.arange(len(cu), device="cuda")
    slot = torch.arange(s["tokens"] // page + 2 * c["n_seq"], device="cuda")
    of = (torch.searchsorted(base, slot, right=True) - 1).clamp(0, c["n_seq"] - 1)
    at = past[of] // page + slot - base[of]
    place = at[:, None] * page + torch.arange(page, device="cuda")          # positions of the slot's rows
    here = place - past[of][:, None] + cu[of][:, None]                      # their tokens
    fresh = (place >= past[of][:, None]) & (here < cu[of + 1][:, None])
    used = fresh.any(1)
    to = torch.where(used, table[of, at.clamp(0, table.shape[1] - 1)], s["n_pages"])
    here = here.clamp(0, max(0, s["tokens"] - 1))
    started = used & (place[:, 0] < past[of])
    for x, codes, scales in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        new = torch.where(fresh[:, :, None, None], x[here], torch.zeros((), device="cuda")).transpose(1, 2)
        before = torch.where(started[:, None], scales[to], torch.zeros((), device="cuda"))
        need = _scale_for(new.abs().amax((2, 3)), fmt)
        scale = torch.where(torch.isnan(before) | torch.isnan(need), float("nan"), torch.maximum(before, need))
        old = _rows(codes, to)
        grown = (scale > before)[:, :, None, None]
        ratio = torch.where(scale > 0, before / scale, torch.zeros_like(scale))[:, :, None, None]
        moved = old.float() * ratio
        moved = moved.round().to(torch.int8) if fmt == INT8 else moved.to(torch.float8_e4m3fn)
        earlier = (started[:, None] & (place < past[of][:, None]))[:, None, :, None]
        raw = torch.where(earlier & grown, moved.view(torch.uint8), old.view(torch.uint8))
        mine = _encode(new, scale[:, :, None, None], fmt).view(torch.uint8)
        codes.view(torch.uint8)[to] = torch.where(fresh[:, None, :, None], mine, raw)
        scales[to] = scale
    return q


def _attn_plain(s):
    c = s["case"]
    n, hkv, dim = c["n_seq"], c["hkv"], c["dim"]
    group = c["hq"] // hkv
    cu, past = s["cu"].long(), s["past"].long()
    i = torch.arange(s["most_new"], device="cuda")
    mine = (cu[:-1, None] + i).clamp(max=max(0, s["tokens"] - 1))
    q = s["q"].float()[mine].view(n, -1, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, dim)
    pages = s["table"].long().clamp(min=0)
    k, v = ((_rows(codes, pages).float() * scales[pages][..., None, None]).transpose(1, 2).reshape(n, hkv, -1, dim)
            for codes, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
    scores = (q @ k.transpose(2, 3)).mul_(dim ** -0.5)
    scores = scores.view(n, hkv, s["most_new"], group, -1)
    seen = torch.arange(scores.shape[-1], device="cuda") <= (past[:, None] + i)[..., None]
    scores.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(n, hkv, -1, p.shape[-1]) @ v).view(n, hkv, s["most_new"], group, dim) / total
    tok, seq, pos = _token_places(s)
    out = out.permute(0, 2, 1, 3, 4)[seq, tok - cu[seq]]
    return out.reshape(s["tokens"], c["hq"], dim).to(s["q"].dtype)


def _weights(x):
    return (x.clamp(0, 1).double() * 2.0 ** WEIGHT_BITS).long()


def _verify_plain(s):
    p, q, n, k = s["p"], s["q"], s["case"]["n_seq"], s["case"]["drafts"]
    row, draft = torch.arange(n, device="cuda"), s["draft"].long()[..., None]
    ok = s["u"][:, :k] * q.gather(2, draft)[..., 0] < p[:, :k].gather(2, draft)[..., 0]
    ok &= torch.arange(k, device="cuda") < s["count"][:, None]
    accepted = ok.long().cumprod(1).sum(1)
    target = p[row, accepted]
    drafted = torch.where((accepted < s["count"])[:, None], q[row, accepted.clamp(max=k - 1)],
                          torch.zeros((), device="cuda"))
    w = _weights(target - drafted)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w, _weights(target))
    total = w.sum(1, keepdim=True)
    limit = torch.minimum((s["u"][:, k:].double() * total.double()).floor().long(), total - 1)
    token = (w.cumsum(1) <= limit).sum(1)
    token = torch.where(total[:, 0] > 0, token, -1)
    return {"accepted": accepted.to(torch.int32), "token": token.to(torch.int32)}


# ---- the package's operators --------------------------------------------------------------------

def _cache(s, gdn):
    if "cache" not in s:
        s["cache"] = gdn.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["cache"]


def _append_own(s, gdn):
    q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    gdn.gdn_kv_append(_cache(s, gdn), s["cu"], s["tokens"], s["past"], s["table"], s["q"], s["k_new"], s["v_new"],
                      s["cos"], s["sin"], s["case"]["interleaved"], q_out)
    return q_out


def _attn_own(s, gdn):
    c, cache = s["case"], _cache(s, gdn)
    if "workspace" not in s:
        size = gdn.gdn_kv_attn_workspace_bytes(cache, c["n_seq"], s["tokens"], c["hq"], s["table"].shape[1])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    gdn.gdn_kv_attn(cache, s["cu"], s["tokens"], s["past"], s["table"], s["q"], c["dim"] ** -0.5, y, s["workspace"])
    return y


def _verify_own(s, gdn):
    accepted, token = (torch.empty(s["case"]["n_seq"], dtype=torch.int32, device="cuda") for _ in range(2))
    gdn.gdn_draft_verify(s["p"], s["q"], s["draft"], s["count"], s["u"], accepted, token)
    return {"accepted": accepted, "token": token}


def run(state):
    op = state["case"]["op"]
    if own:
        import gated_deltanet_linear_pre_gb300 as gdn
        out = {"append": _append_own, "attn": _attn_own, "verify": _verify_own}[op](state, gdn)
    else:
        out = {"append": _append_plain, "attn": _attn_plain, "verify": _verify_plain}[op](state)
    if op != "append":
        return out
    # the cache itself, without the spare page.  An int8 code is a whole number of its page's scale, and a
    # float8 code a value in units of it: both forms agree on every one
    n = state["n_pages"]
    return {"q": out, "k": state["k"][:n], "v": state["v"][:n],
            "k_scale": state["k_scale"][:n], "v_scale": state["v_scale"][:n]}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_append(s):
    """Sequence by sequence and page by page; the codes of int8 pages are whole numbers (no value in 64 bits)."""
    c = s["case"]
    cu, past, table = s["cu"].tolist(), s["past"].tolist(), s["table"].tolist()
    page, fmt, half = c["page"], c["fmt"], c["rot"] // 2
    top = 127.0 if fmt == INT8 else 448.0

    def turned(x, pos):
        x = x.double()
        if not half:
            return x
        y = x.clone()
        i = torch.arange(half, device="cuda")
        ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        co, si = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
        y[..., ia] = x[..., ia] * co - x[..., ib] * si
        y[..., ib] = x[..., ia] * si + x[..., ib] * co
        return y

    # positions by a host loop over sequences, apart from the plain form's search
    pos = torch.tensor([past[i] + j for i in range(c["n_seq"]) for j in range(cu[i + 1] - cu[i])], device="cuda",
                       dtype=torch.long)
    q, k, v = turned(s["q"], pos), turned(s["k_new"], pos), s["v_new"].double()
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        codes, scales = s[name].clone(), s[name + "_scale"].double()
        for i in range(c["n_seq"]):
            first, last = past[i], past[i] + cu[i + 1] - cu[i]
            for pg in range(first // page, -(-last // page) if last > first else 0):
                lo, hi = max(first, pg * page), min(last, (pg + 1) * page)
                new = x[cu[i] + lo - first:cu[i] + hi - first].transpose(0, 1)       # [heads, rows, dim]
                need = new.abs().amax((1, 2)) / top
                need = torch.where(need > 0, torch.exp2(torch.ceil(torch.log2(need))).clamp(min=2.0 ** -100), 0.0)
                at = table[i][pg]
                keep = lo - pg * page
                if keep:
                    before = scales[at]
                    now = torch.maximum(before, need)
                    moved = codes[at, :, :keep].float().double() * (before / now.clamp(min=2.0 ** -100))[:, None, None]
                    codes[at, :, :keep] = (moved.round() if fmt == INT8 else moved).to(torch.float32).to(codes.dtype)
                else:
                    now = need
                mine = new / now.clamp(min=2.0 ** -100)[:, None, None]
                codes[at, :, keep:hi - pg * page] = (mine.round() if fmt == INT8 else mine).to(codes.dtype)
                scales[at] = now
        n = s["n_pages"]
        out[name] = None if fmt == INT8 else codes[:n].float().double()
        out[name + "_scale"] = scales[:n]
    return out


def _exact_attn(s):
    c = s["case"]
    cu, past, page, dim = s["cu"].tolist(), s["past"].tolist(), c["page"], c["dim"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["n_seq"]):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        held = past[i] + b - a
        ids = s["table"][i, :-(-held // page)].long()
        for h in range(c["hkv"]):
            k, v = ((s[x].view(torch.uint8)[ids, h].view(s[x].dtype).double()
                     * s[x + "_scale"][ids, h].double()[:, None, None]).reshape(-1, dim)[:held] for x in ("k", "v"))
            for lo in range(a, b, 512):
                hi = min(b, lo + 512)
                q = s["q"][lo:hi, h * group:(h + 1) * group].double()
                x = torch.einsum("tgd,nd->tgn", q, k) / dim ** 0.5
                late = torch.arange(held, device="cuda")[None] > past[i] + torch.arange(lo - a, hi - a, device="cuda")[:, None]
                x = torch.softmax(x.masked_fill(late[:, None], float("-inf")), -1)
                out[lo:hi, h * group:(h + 1) * group] = torch.einsum("tgn,nd->tgd", x, v)
    return out


def _exact_verify(s):
    """Whole numbers: the rule written out sequence by sequence, with sums in 64 bits."""
    k = s["case"]["drafts"]
    u, count, draft = s["u"].tolist(), s["count"].tolist(), s["draft"].tolist()
    accepted, token = [], []
    for i in range(s["case"]["n_seq"]):
        a = 0
        while a < count[i] and u[i][a] * float(s["q"][i, a, draft[i][a]]) < float(s["p"][i, a, draft[i][a]]):
            a += 1
        p = s["p"][i, a].double()
        r = (p - s["q"][i, a].double()).clamp(min=0) if a < count[i] else p
        r = r if float(r.sum()) > 0 else p
        sums = r.cumsum(0)
        accepted.append(a)
        token.append(min(int((sums <= u[i][k] * float(sums[-1])).sum()), len(sums) - 1))
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"accepted": torch.tensor(accepted, **i32), "token": torch.tensor(token, **i32)}


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify}[case["op"]](s)
