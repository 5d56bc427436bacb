"""GPU parity of the paged 8-bit cache: gdn_kv_append against the rotation's and the quantisation's
definitions, gdn_kv_attn against softmax attention in 64 bits (tests/kv_util.py), over ragged batches,
page ends inside a tile, odd groups of heads, idle slots, missing pages and values that are not finite."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()


class Batch:
    """A pool of pages filled with garbage, a table, and new tokens."""

    def __init__(self, new, past, hq, heads, dim, page, fmt, dtype, seed=0, rot=None, interleaved=False, scale=1.0):
        import gated_deltanet_linear_pre_gb300 as gdn
        import kv_util as u
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.past_h, self.page, self.fmt, self.dtype = list(new), list(past), page, fmt, dtype
        self.heads, self.hq, self.dim = heads, hq, dim
        self.cu_h = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.T = int(self.cu_h[-1])
        self.table_h, n_pages = u.page_table(new, past, page, seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cu, self.past = torch.tensor(self.cu_h, **i32), torch.tensor(self.past_h, **i32)
        self.table = torch.tensor(self.table_h, **i32)
        shape = (n_pages, heads, page, dim)
        raw = [torch.randint(0, 256, shape, device="cuda", generator=g, dtype=torch.int32).to(torch.uint8) for _ in range(2)]
        self.k, self.v = (r.view(u.CODES[fmt]) for r in raw)
        self.ks, self.vs = (torch.full((n_pages, heads), float("nan"), device="cuda") for _ in range(2))
        dt = u.TYPES[dtype]
        qkv = torch.randn((self.T, hq + 2 * heads, dim), device="cuda", generator=g) * scale
        self.qkv = qkv.to(dt)
        self.q, self.kn, self.vn = self.qkv[:, :hq], self.qkv[:, hq:hq + heads], self.qkv[:, hq + heads:]
        rot = dim if rot is None else rot
        self.cos = self.sin = None
        if rot:
            ang = torch.arange(max(1, max(a + b for a, b in zip(new, past))), device="cuda").double()[:, None] * \
                10000.0 ** (-torch.arange(rot // 2, device="cuda").double() / (rot // 2))
            self.cos, self.sin = ang.cos().float(), ang.sin().float()
        self.interleaved = interleaved
        self.cache = gdn.kv_cache(self.k, self.v, self.ks, self.vs)

    def fill_past(self, seed=1):
        """Codes and scales as earlier calls leave them, at every position before the new tokens."""
        import kv_util as u
        g = torch.Generator(device="cuda").manual_seed(seed)
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            x = torch.randn(codes.shape, device="cuda", generator=g)
            new = (x * 30).round().clamp(-127, 127).to(torch.int8) if self.fmt == "int8" else (x * 60).to(torch.float8_e4m3fn)
            sc = torch.exp2(torch.randint(-1, 2, scales.shape, device="cuda", generator=g).float() - (5 if self.fmt == "int8" else 6))
            for s, past in enumerate(self.past_h):
                for at in range(-(-max(0, past) // self.page)):
                    rows = min(self.page, past - at * self.page)
                    pg = int(self.table_h[s, at])
                    codes.view(torch.uint8)[pg, :, :rows] = new.view(torch.uint8)[pg, :, :rows]
                    scales[pg] = sc[pg]

    def append(self, q_out=None, stream=None):
        import gated_deltanet_linear_pre_gb300 as gdn
        q_out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda") if q_out is None else q_out
        gdn.gdn_kv_append(self.cache, self.cu, self.T, self.past, self.table, self.q, self.kn, self.vn, self.cos,
                          self.sin, self.interleaved, q_out, stream)
        return q_out

    def attend(self, q=None, softmax_scale=None, workspace=None):
        import gated_deltanet_linear_pre_gb300 as gdn
        q = self.q if q is None else q
        n, width = self.table.shape
        size = gdn.gdn_kv_attn_workspace_bytes(self.cache, n, self.T, self.hq, width)
        ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda") if workspace is None else workspace
        guard = 32
        buf = torch.full((self.T * self.hq * self.dim + 2 * guard,), 7.0, dtype=q.dtype, device="cuda")
        y = buf[guard:buf.numel() - guard].view(self.T, self.hq, self.dim)
        gdn.gdn_kv_attn(self.cache, self.cu, self.T, self.past, self.table, q,
                        self.dim ** -0.5 if softmax_scale is None else softmax_scale, y, ws[:size])
        if size:
            gdn.gdn_kv_attn_check(ws)
        torch.cuda.synchronize()
        assert bool((buf[:guard] == 7).all()) and bool((buf[-guard:] == 7).all()), "output written outside y"
        if workspace is None:
            assert bool((ws[size:] == 0xA5).all()), "workspace overrun"
        return y

    def reference(self, q=None, softmax_scale=None):
        import kv_util as u
        with np.errstate(invalid="ignore"):
            return u.attention(u.values(self.q if q is None else q), u.values(self.k), u.values(self.v), u.values(self.ks),
                               u.values(self.vs), self.table_h, self.cu_h, self.past_h, self.page,
                               self.dim ** -0.5 if softmax_scale is None else softmax_scale)


def check_attention(b, q=None, softmax_scale=None, dtype=None):
    import kv_util as u
    y = u.values(b.attend(q, softmax_scale))
    ref, wabs, xabs = b.reference(q, softmax_scale)
    bound = u.attention_bound(ref, wabs, xabs, dtype or b.dtype)
    bad = ~(np.abs(y - ref) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst {np.nanmax(np.abs(y - ref) / bound)} times the bound"


# ---- the append -------------------------------------------------------------------------------------

def stored(b, s):
    """Values [past + new, heads, d] of sequence s, k and v."""
    import kv_util as u
    held = b.past_h[s] + b.new[s]
    return (u.dense(u.values(b.k), u.values(b.ks), b.table_h, s, held, b.page)[0],
            u.dense(u.values(b.v), u.values(b.vs), b.table_h, s, held, b.page)[0])


def check_scales(b, x, scales, upto):
    """Every touched page's scale is the power of two that its values need.  x [T, h, d] in 64 bits; the
    rotation's fp32 roundings (three, of 2^-24 of at most twice the largest channel) leave the maximum
    uncertain by 2^-21 of it."""
    import kv_util as u
    for s in range(len(b.new)):
        for at in range(-(-upto[s] // b.page)):
            lo, hi = at * b.page, min(upto[s], (at + 1) * b.page)
            rows = slice(b.cu_h[s] + lo - b.past_h[s], b.cu_h[s] + hi - b.past_h[s])
            amax = np.abs(x[rows]).max(axis=(0, 2))
            sc = u.values(scales)[b.table_h[s, at]]
            assert np.all(np.exp2(np.round(np.log2(sc))) == sc)
            assert np.all(sc * u.QMAX[b.fmt] >= amax * (1 - 2.0 ** -21))
            assert np.all(sc / 2 * u.QMAX[b.fmt] <= amax * (1 + 2.0 ** -21))


SHAPES = [  # new, hq, heads, dim, page
    ([1], 3, 1, 128, 16),
    ([5, 0, 1, 70], 6, 2, 64, 32),
    ([40, 129, 3], 8, 8, 128, 64),
    ([300], 4, 4, 64, 128),
    ([1] * 70, 2, 1, 128, 16),
]


@pytest.mark.parametrize("new,hq,heads,dim,page", SHAPES)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rot,interleaved", [(None, False), (32, True), (32, False), (0, False), (None, True)])
def test_append_from_empty(new, hq, heads, dim, page, fmt, dtype, rot, interleaved):
    import kv_util as u
    b = Batch(new, [0] * len(new), hq, heads, dim, page, fmt, dtype, seed=len(new), rot=rot, interleaved=interleaved)
    q_out = u.values(b.append())
    pos = u.positions(b.cu_h, b.past_h)
    cos, sin = (None, None) if b.cos is None else (u.values(b.cos), u.values(b.sin))
    q, k, v = (u.rotate(u.values(t), pos, cos, sin, interleaved) for t in (b.q, b.kn, b.vn))
    v = u.values(b.vn)
    # three fp32 roundings of terms of at most the row's largest, then the type's own
    big = np.abs(u.values(b.q)).max(axis=-1, keepdims=True)
    assert np.all(np.abs(q_out - q) <= u.UNIT[dtype] * np.abs(q) + big * 2.0 ** -22 + 2.0 ** -25)
    check_scales(b, k, b.ks, new)
    check_scales(b, v, b.vs, new)
    for s in range(len(new)):
        rows = slice(b.cu_h[s], b.cu_h[s + 1])
        for got, x, scales in zip(stored(b, s), (k[rows], v[rows]), (b.ks, b.vs)):
            sc = u.values(scales)[b.table_h[s][np.arange(new[s]) // page]].reshape(new[s], heads, 1)
            # half a step: of the integers, or of a 3-bit mantissa above the smallest normal 2^-6
            step = sc / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
            # (the rounded value may lie past the half by the rotation's own 2^-21)
            assert np.all(np.abs(got - x) <= step * (1 + 2.0 ** -6) + np.abs(x).max(initial=0) * 2.0 ** -21)


MANY = [400, 1, 333, 0, 390, 17, 256]  # more pages and heads than a wave of blocks, as one call


@pytest.mark.parametrize("dim,page", [(128, 16), (64, 16), (64, 32), (128, 32), (64, 128)])
@pytest.mark.parametrize("fmt,dtype,rot,interleaved", [("int8", "bf16", None, False), ("e4m3", "fp16", 32, True)])
def test_append_many_pages(dim, page, fmt, dtype, rot, interleaved):
    """A large call's pages against the definitions; the same tokens stored a sequence at a time, behind
    pages that are partly filled, give the same codes and scales bit for bit."""
    test_append_from_empty(MANY, 16, 16, dim, page, fmt, dtype, rot, interleaved)
    import gated_deltanet_linear_pre_gb300 as gdn
    one, each = (Batch(MANY, [5, 0, 1000, 3, 16, 31, 127], 16, 16, dim, page, fmt, dtype, seed=9, rot=rot, interleaved=interleaved)
                 for _ in range(2))
    for b in (one, each):
        b.fill_past()
    q_out = one.append()
    q_each = torch.full_like(q_out, float("nan"))
    for s, n in enumerate(MANY):
        rows = slice(int(each.cu_h[s]), int(each.cu_h[s + 1]))
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        gdn.gdn_kv_append(each.cache, cu, n, each.past[s:s + 1], each.table[s:s + 1], each.q[rows], each.kn[rows], each.vn[rows],
                          each.cos, each.sin, interleaved, q_each[rows])
    assert torch.equal(q_out, q_each)
    for a, b in ((one.k, each.k), (one.v, each.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in ((one.ks, each.ks), (one.vs, each.vs)):
        assert torch.equal(a.nan_to_num(3), b.nan_to_num(3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64)])
def test_append_in_pieces_stays_below_one_step(fmt, dim, page):
    """A page filled by many calls, each with larger values than the last: every growth rounds again, and
    the error stays below one step of the final scale; the scale is that of one call."""
    import gated_deltanet_linear_pre_gb300 as gdn
    import kv_util as u
    total, cuts = 2 * page + 5, [1, 1, 2, 3, 1, 8]
    whole = Batch([total], [0], 2, 2, dim, page, fmt, "fp16", seed=3, rot=0)
    grow = torch.exp2(torch.linspace(0, 7, total, device="cuda"))[:, None, None]
    whole.qkv.copy_((whole.qkv.float() * grow / 16).to(torch.float16))
    whole.append()
    parts = Batch([total], [0], 2, 2, dim, page, fmt, "fp16", seed=3, rot=0)
    parts.qkv.copy_(whole.qkv)
    at = i = 0
    while at < total:
        n = min(cuts[i % len(cuts)], total - at)
        i += 1
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        gdn.gdn_kv_append(parts.cache, cu, n, torch.tensor([at], dtype=torch.int32, device="cuda"), parts.table, None,
                          parts.kn[at:at + n], parts.vn[at:at + n], None, None, False, None)
        at += n
    used = parts.table_h[0, :3]
    assert torch.equal(parts.ks[used], whole.ks[used]) and torch.equal(parts.vs[used], whole.vs[used])
    for got, x, scales in zip(stored(parts, 0), (parts.kn, parts.vn), (parts.ks, parts.vs)):
        x = u.values(x)
        sc = u.values(scales)[parts.table_h[0][np.arange(total) // page]].reshape(total, 2, 1)
        # e4m3: growth by powers of two only rounds below 2^-6 of the scale, to half a step of 2^-9 each time
        step = sc if fmt == "int8" else np.abs(x) * 2.0 ** -4 + sc * 2.0 ** -9
        assert np.all(np.abs(got - x) < step)


def test_append_leaves_other_places_alone():
    b = Batch([3, 20], [13, 30], 2, 2, 128, 16, "int8", "bf16", seed=5)
    b.fill_past()
    before = b.k.clone(), b.ks.clone()
    b.append()
    touched = {int(b.table_h[0, 0]), *(int(x) for x in b.table_h[1, 1:4])}
    for pg in range(b.k.shape[0]):
        if pg not in touched:
            assert torch.equal(b.k[pg], before[0][pg]), pg
            assert torch.equal(b.ks[pg].nan_to_num(3), before[1][pg].nan_to_num(3)), pg
    # rows behind the last new one in the last page
    last, rows = int(b.table_h[1, 3]), (30 + 20) % 16
    assert torch.equal(b.k[last, :, rows:], before[0][last, :, rows:])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_values_that_are_not_finite(fmt):
    """An infinity or NaN makes its page and head's scale NaN, for good, and no other's."""
    import kv_util as u
    b = Batch([40], [0], 2, 2, 64, 16, fmt, "fp16", rot=0)
    b.kn[3, 0, 5] = float("inf")
    b.vn[20, 1, 63] = float("nan")
    b.append()
    ks, vs = u.values(b.ks)[b.table_h[0, :3]], u.values(b.vs)[b.table_h[0, :3]]
    assert np.array_equal(np.isnan(ks), [[True, False], [False, False], [False, False]])
    assert np.array_equal(np.isnan(vs), [[False, False], [False, True], [False, False]])
    y = u.values(b.attend())
    assert np.isnan(y[:, 0]).all() and not np.isnan(y[:16, 1]).any()
    assert np.isnan(y[20:, 1]).all()


def test_append_zeros_and_tiny_values():
    import kv_util as u
    b = Batch([16, 16], [0, 0], 1, 1, 64, 16, "int8", "bf16", rot=0)
    b.qkv[:16] = 0
    b.qkv[16:] = 1e-38
    b.append()
    assert float(b.ks[b.table_h[0, 0], 0]) == 0.0
    assert float(b.ks[b.table_h[1, 0], 0]) == 2.0 ** -100
    assert not stored(b, 0)[0].any() and not stored(b, 1)[0].any()
    assert not u.values(b.attend()).any()


def test_append_refuses_nothing_it_can_skip():
    """Idle slots (negative positions), positions past the table and bad entries store nothing."""
    b = Batch([2, 3, 4], [-2, 30, 14], 2, 1, 128, 16, "e4m3", "bf16")
    b.table[1, 1] = 10 ** 6
    b.table[2] = -7
    before = b.k.clone().view(torch.uint8), b.ks.clone()
    small = b.table[:, :2].contiguous()
    import gated_deltanet_linear_pre_gb300 as gdn
    q_out = torch.full(b.q.shape, float("nan"), dtype=b.q.dtype, device="cuda")
    gdn.gdn_kv_append(b.cache, b.cu, b.T, b.past, small, b.q, b.kn, b.vn, b.cos, b.sin, False, q_out)
    torch.cuda.synchronize()
    assert torch.equal(b.k.view(torch.uint8), before[0]) and torch.equal(b.ks.nan_to_num(3), before[1].nan_to_num(3))
    assert not bool(q_out.isnan().any())


# ---- the attention ------------------------------------------------------------------------------------

CASES = [  # new, past, hq, heads, dim, page
    ([1], [0], 1, 1, 128, 16),
    ([1], [300], 6, 2, 128, 16),
    ([1, 1, 1, 1, 1], [0, 15, 16, 63, 1000], 8, 1, 64, 16),
    ([1] * 9, [5, 250, 1, 0, 64, 127, 128, 700, 33], 12, 4, 128, 64),
    ([3, 0, 5, 1], [7, 90, 0, 600], 10, 2, 128, 32),
    ([6, 2, 6], [1000, 3, 77], 16, 2, 64, 128),
    ([1, 40, 1], [90, 30, 2000], 14, 2, 128, 64),
    ([130, 7], [0, 259], 3, 1, 128, 32),
    ([97], [4], 4, 4, 64, 16),
    ([1], [5000], 64, 1, 128, 64),
    ([300, 1, 2, 200], [0, 900, 40, 1000], 8, 2, 128, 64),
    ([260, 129], [130, 0], 4, 4, 64, 128),
    ([70, 5, 90], [513, 1200, 126], 48, 1, 128, 16),
]


@pytest.mark.parametrize("new,past,hq,heads,dim,page", CASES)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attention(new, past, hq, heads, dim, page, fmt, dtype):
    b = Batch(new, past, hq, heads, dim, page, fmt, dtype, seed=sum(past) + len(new), scale=2.0)
    b.fill_past()
    b.append()
    check_attention(b)


def test_attention_of_many_sequences():
    """More sequences than a block has threads."""
    rng = np.random.default_rng(4)
    new, past = rng.integers(0, 3, 600).tolist(), rng.integers(0, 60, 600).tolist()
    b = Batch(new, past, 4, 2, 64, 16, "e4m3", "fp16", seed=9)
    b.fill_past()
    b.append()
    check_attention(b)


def test_attention_rows_that_see_nothing():
    import kv_util as u
    b = Batch([2, 3, 4, 5], [-2, -1, 14, 40], 4, 2, 128, 16, "int8", "fp16")
    b.fill_past()
    b.append()
    b.table_h[2] = -1                       # a sequence without a page
    b.table_h[3, 1] = b.k.shape[0]          # a hole in the middle of one
    b.table.copy_(torch.tensor(b.table_h))
    y = u.values(b.attend())
    assert not y[:2].any() and not y[2].any() and not y[5:9].any()
    check_attention(b)


def test_attention_peaked_scores_and_uneven_pages():
    """Scores of several hundred, and pages whose v differ by 2^10 in size."""
    b = Batch([4, 1], [500, 300], 8, 2, 128, 32, "int8", "fp16", seed=2, scale=12.0)
    b.fill_past()
    b.append()
    sizes = torch.exp2(torch.randint(-10, 1, b.vs.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).float())
    b.vs.mul_(sizes)
    check_attention(b)
    check_attention(b, softmax_scale=0.0)
    check_attention(b, softmax_scale=-0.05)


def test_attention_bf16_queries_beyond_fp16():
    b = Batch([1, 1], [40, 90], 4, 2, 64, 16, "e4m3", "bf16", seed=6)
    b.fill_past()
    b.append()
    q = b.q.clone()
    q[0] *= 1e30
    q[1] *= 1e-30
    check_attention(b, q=q, softmax_scale=1e-30)


# ---- the prompt way: sequences of more than 128 query rows ------------------------------------------------

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_scales_of_either_sign_and_uneven_pages(fmt, dtype, dim):
    """Pages whose k and v differ by 2^8 in size, scores of several hundred, scales of 0 and below."""
    b = Batch([70, 1, 150], [100, 600, 0], 8, 2, dim, 32, fmt, dtype, seed=2, scale=6.0)
    b.fill_past()
    b.append()
    g = torch.Generator("cuda").manual_seed(1)
    for scales in (b.ks, b.vs):
        scales.mul_(torch.exp2(torch.randint(-8, 1, scales.shape, device="cuda", generator=g).float()))
    for softmax_scale in (0.1, -0.1, 0.0):
        check_attention(b, softmax_scale=softmax_scale)


def test_prompt_pages_that_are_missing_zero_or_not_finite():
    """A hole in the table, a page of zeros, and a NaN page: only rows that see it are NaN."""
    import kv_util as u
    b = Batch([80, 80, 80], [300, 300, 300], 4, 2, 128, 64, "int8", "fp16", seed=4)
    b.fill_past()
    b.append()
    b.table_h[0, 1] = -1
    b.table_h[0, 3] = 10 ** 6
    b.table.copy_(torch.tensor(b.table_h))
    zero, bad = int(b.table_h[1, 2]), int(b.table_h[2, 5])
    for t in (b.k, b.v, b.ks, b.vs):
        t[zero] = 0
    check_attention(b)
    b.vs[bad, 1] = float("nan")                       # positions 320 onwards of the last sequence
    y = u.values(b.attend())
    assert np.isnan(y[160 + 20:, 2:]).all() and not np.isnan(y[:, :2]).any() and not np.isnan(y[:160]).any()


def test_prompt_queries_at_the_ends_of_their_types():
    for dtype, size, softmax_scale in (("bf16", 1e30, 1e-30), ("bf16", 1e-30, 1e30), ("fp16", 3e4, 1e-5)):
        b = Batch([90], [40], 4, 2, 64, 16, "e4m3", dtype, seed=6, rot=0)
        b.fill_past()
        b.append()
        q = torch.randn(b.q.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).clamp(-2, 2)
        check_attention(b, q=(q * size).to(b.q.dtype), softmax_scale=softmax_scale)


def test_prompts_among_empty_and_single_token_sequences():
    """More long sequences than a batch without empty ones could hold: some take the step kernel."""
    new = [0] * 60 + [40, 0, 200, 1, 1, 0, 180, 33] + [0] * 60
    past = [7] * len(new)
    past[62] = -30                                    # begins before position 0
    b = Batch(new, past, 16, 2, 128, 32, "e4m3", "bf16", seed=8)
    b.fill_past()
    b.append()
    check_attention(b)


@pytest.mark.parametrize("new,past,hq,heads,dim,page", [
    # more units than CTAs: handed out one by one
    ([700, 333], [0, 0], 64, 16, 64, 64),
    ([333, 40, 1, 300], [30, 0, 500, 100], 128, 32, 64, 16),
    # the next prompt is many sequences away, single tokens and none between
    ([70] + [1] * 33 + [0, 1, 90] + [1] * 70 + [45], [100] + [9] * 107, 8, 2, 128, 32),
    # more sequences than a block has threads
    ([1] * 290 + [60] * 4, [3] * 294, 4, 1, 64, 16),
    # a few long units: cut
    ([40, 1, 90], [9000, 5, 4000], 8, 2, 128, 64),
    ([140], [3000], 16, 1, 64, 128),
])
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16")])
def test_prompt_units_handed_out_or_cut(new, past, hq, heads, dim, page, fmt, dtype):
    b = Batch(new, past, hq, heads, dim, page, fmt, dtype, seed=len(new))
    b.fill_past()
    b.append()
    check_attention(b)
    again = b.attend().clone()
    assert torch.equal(b.attend(), again)             # whichever CTA takes a unit


def test_prompt_units_handed_out_past_one_without_images():
    """The middle prompt has a hole in its table and takes the other way; its place is passed over."""
    b = Batch([200, 300, 250], [0, 60, 0], 32, 8, 128, 32, "e4m3", "bf16", seed=2)
    b.fill_past()
    b.append()
    b.table_h[1, 2] = -1
    b.table.copy_(torch.tensor(b.table_h))
    check_attention(b)


@pytest.mark.parametrize("hole", [0, 1, 2, 3])
def test_prompt_ranges_that_begin_in_a_sequence_without_images(hole):
    """A range of cut units may begin with units that have no images: what it has of the next sequence's
    first unit is still its second part."""
    b = Batch([192, 378, 35, 106, 1], [1167, 0, 214, 15, 127], 28, 4, 128, 16, "int8", "bf16", seed=7)
    b.fill_past()
    b.append()
    b.table_h[hole, 5] = -1
    b.table.copy_(torch.tensor(b.table_h))
    check_attention(b)


def test_prompts_repeat_exactly_and_follow_their_lengths_in_a_graph():
    import gated_deltanet_linear_pre_gb300 as gdn
    b = Batch([150, 1, 90], [700, 300, 10], 8, 2, 128, 64, "int8", "bf16", seed=7)
    b.fill_past()
    b.append()
    size = gdn.gdn_kv_attn_workspace_bytes(b.cache, 3, b.T, b.hq, b.table.shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.empty(b.q.shape, dtype=b.q.dtype, device="cuda")
    graph = torch.cuda.CUDAGraph()
    call = lambda: gdn.gdn_kv_attn(b.cache, b.cu, b.T, b.past, b.table, b.q, 0.1, y, ws)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for cuts, past in (([150, 1, 90], [700, 300, 10]), ([1, 239, 1], [849, 62, 99]), ([80, 81, 80], [0, 0, 20]), ([0, 0, 241], [9, 9, -141])):
        b.new, b.past_h, b.cu_h = cuts, past, np.concatenate([[0], np.cumsum(cuts)])
        b.cu.copy_(torch.tensor(b.cu_h))
        b.past.copy_(torch.tensor(past))
        graph.replay()
        gdn.gdn_kv_attn_check(ws)
        replayed = y.clone()
        assert torch.equal(b.attend(softmax_scale=0.1), replayed)
        check_attention(b, softmax_scale=0.1)


def test_attention_ignores_what_no_query_sees():
    """Scales and codes of unused pages and of rows past the end are whatever they were."""
    b = Batch([1, 2], [37, 130], 4, 1, 128, 64, "e4m3", "bf16", seed=8)
    b.fill_past()
    b.append()
    y0 = b.attend().clone()
    used = {int(b.table_h[s, at]) for s in range(2) for at in range(-(-(b.past_h[s] + b.new[s]) // 64))}
    for pg in range(b.k.shape[0]):
        if pg not in used:
            b.ks[pg], b.vs[pg] = float("inf"), float("nan")
    for s in range(2):
        held = b.past_h[s] + b.new[s]
        pg, rows = int(b.table_h[s, (held - 1) // 64]), (held - 1) % 64 + 1
        for codes in (b.k, b.v):
            codes.view(torch.uint8)[pg, :, rows:] = 0x7F
    assert torch.equal(b.attend(), y0)


def test_attention_is_the_same_every_time_and_in_a_workspace_of_any_content():
    import gated_deltanet_linear_pre_gb300 as gdn
    b = Batch([1, 3, 1], [3000, 10, 700], 8, 2, 128, 64, "e4m3", "fp16", seed=1)
    b.fill_past()
    b.append()
    y = b.attend().clone()
    size = gdn.gdn_kv_attn_workspace_bytes(b.cache, 3, b.T, b.hq, b.table.shape[1])
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(b.attend(workspace=ws), y)


def test_strided_and_cut_inputs():
    """Queries and table rows with strides of their own give what dense ones give."""
    b = Batch([2, 9], [20, 100], 6, 2, 128, 16, "int8", "bf16", seed=3)
    b.fill_past()
    dense_q = b.append()
    y = b.attend(q=dense_q).clone()
    wide = torch.zeros((b.T, 9, 128), dtype=b.q.dtype, device="cuda")
    wide[:, 2:8] = dense_q
    assert torch.equal(b.attend(q=wide[:, 2:8]), y)
    table = torch.full((2, b.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    kept, b.table = b.table, table[:, :b.table.shape[1]]
    assert torch.equal(b.attend(q=dense_q), y)
    b.table = kept


@pytest.mark.parametrize("hq,heads", [(6, 2), (64, 1)])
def test_tokens_far_apart(hq, heads):
    """Two tokens 2^30 elements and more apart, as single rows and as rows enough for the prompts' kernels, give what
    dense ones give."""
    b = Batch([2], [100], hq, heads, 128, 16, "int8", "bf16", seed=3)
    b.fill_past()
    codes = [t.clone() for t in (b.k, b.v, b.ks, b.vs)]
    q = b.append()
    y, stored = b.attend(q=q).clone(), [t.clone() for t in (b.k, b.v, b.ks, b.vs)]
    for t, was in zip((b.k, b.v, b.ks, b.vs), codes):
        t.copy_(was)
    row, far = (hq + 2 * heads) * 128, (1 << 30) + 64
    wide = torch.empty(far + row, dtype=b.q.dtype, device="cuda").as_strided((2, hq + 2 * heads, 128), (far, 128, 1))
    wide.copy_(b.qkv)
    b.q, b.kn, b.vn = wide[:, :hq], wide[:, hq:hq + heads], wide[:, hq + heads:]
    assert torch.equal(b.append(q_out=torch.empty_like(q)), q)
    for t, was in zip((b.ks, b.vs), stored[2:]):
        assert torch.equal(t.nan_to_num(-1.0), was.nan_to_num(-1.0))
    assert torch.equal(b.k, stored[0]) and torch.equal(b.v, stored[1])
    wide[:, :hq] = q
    assert torch.equal(b.attend(q=wide[:, :hq]), y)


def test_long_cache_offsets_past_32_bits():
    """Pages whose byte offset does not fit 32 bits."""
    import kv_util as u
    heads, page, dim = 8, 128, 128
    n_pages = (1 << 32) // (heads * page * dim) + 40
    import gated_deltanet_linear_pre_gb300 as gdn
    b = Batch([1], [300], 8, heads, dim, page, "int8", "fp16", seed=2)
    b.k, b.v = (torch.zeros((n_pages, heads, page, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    b.ks, b.vs = (torch.zeros((n_pages, heads), device="cuda") for _ in range(2))
    b.table_h[0, :3] = [n_pages - 1, 7, n_pages - 3]
    b.table.copy_(torch.tensor(b.table_h))
    b.cache = gdn.kv_cache(b.k, b.v, b.ks, b.vs)
    for at in range(3):
        pg = int(b.table_h[0, at])
        b.k[pg] = torch.randint(-127, 128, b.k[pg].shape, device="cuda").to(torch.int8)
        b.v[pg] = torch.randint(-127, 128, b.v[pg].shape, device="cuda").to(torch.int8)
        b.ks[pg], b.vs[pg] = 2.0 ** -6, 2.0 ** -5
    b.append()
    y = u.values(b.attend())
    # the reference on the three pages alone
    sel = [int(x) for x in b.table_h[0, :3]]
    table = np.array([[0, 1, 2]], np.int32)
    ref, wabs, xabs = u.attention(u.values(b.q), *(u.values(t[sel]) for t in (b.k, b.v, b.ks, b.vs)), table, b.cu_h, b.past_h,
                                  page, dim ** -0.5)
    assert np.all(np.abs(y - ref) <= u.attention_bound(ref, wabs, xabs, "fp16"))


def test_side_stream_and_graph_replay_with_new_lengths():
    """A captured append and attention follow the lengths, tokens and tables that the buffers then hold."""
    import gated_deltanet_linear_pre_gb300 as gdn
    b = Batch([1, 1, 1], [200, 20, 90], 8, 2, 128, 32, "int8", "fp16", seed=5)
    b.fill_past()
    size = gdn.gdn_kv_attn_workspace_bytes(b.cache, 3, b.T, b.hq, b.table.shape[1])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    q_rot, y = (torch.empty((b.T, b.hq, b.dim), dtype=b.q.dtype, device="cuda") for _ in range(2))

    def both():
        b.append(q_rot)
        gdn.gdn_kv_attn(b.cache, b.cu, b.T, b.past, b.table, q_rot, 0.1, y, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for past in ([200, 20, 90], [3, 20, -1], [0, 0, 50]):
        b.past.copy_(torch.tensor(past))
        b.qkv.copy_(torch.randn_like(b.qkv))
        codes = [t.clone() for t in (b.k.view(torch.uint8), b.v.view(torch.uint8), b.ks, b.vs)]
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        for t, c in zip((b.k.view(torch.uint8), b.v.view(torch.uint8), b.ks, b.vs), codes):
            t.copy_(c)
        both()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
        b.past_h = past
        check_attention(b, q=q_rot, softmax_scale=0.1)


def test_empty_calls():
    b = Batch([0, 0], [5, 0], 2, 1, 64, 16, "int8", "fp16")
    b.append()
    assert b.attend().numel() == 0


# ---- refusals -------------------------------------------------------------------------------------------

def test_binding_refusals():
    import gated_deltanet_linear_pre_gb300 as gdn
    b = Batch([2, 1], [5, 40], 4, 2, 64, 16, "int8", "fp16")
    n, width = b.table.shape
    size = gdn.gdn_kv_attn_workspace_bytes(b.cache, n, b.T, b.hq, width)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = torch.empty(b.q.shape, dtype=b.q.dtype, device="cuda")
    attn = lambda **k: gdn.gdn_kv_attn(b.cache, b.cu, b.T, b.past, k.get("table", b.table), k.get("q", b.q), 0.1,
                                       k.get("y", y), k.get("ws", ws))
    with pytest.raises(gdn.GdnError) as e:
        attn(ws=ws[:size - 1])
    assert e.value.status == 4
    with pytest.raises(TypeError):
        attn(q=b.q.float())
    with pytest.raises(ValueError):
        attn(q=b.q.transpose(1, 2))
    with pytest.raises(ValueError):
        attn(table=b.table[:1])
    with pytest.raises(TypeError):
        attn(y=y.to(torch.bfloat16))
    with pytest.raises(gdn.GdnError) as e:
        attn(y=b.qkv.view(-1)[:y.numel()].view(y.shape))
    assert e.value.status == 1 and "overlaps" in str(e.value)
    with pytest.raises(TypeError):
        gdn.kv_cache(b.k.to(torch.int16), b.v, b.ks, b.vs)
    with pytest.raises(ValueError):
        gdn.kv_cache(b.k, b.v, b.ks[:, :1], b.vs)
